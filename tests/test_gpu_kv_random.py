"""Seeded random problems of the 4-bit cache: shapes, types, page sizes, ragged batches with empty sequences, masks,
strides, expected lengths and pieces drawn at random, against the 64-bit reference."""
import random

import pytest
import torch

import _kv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def wq():
    import weight_only_quantized_w4a16_amd as m
    m.lib()
    assert torch.cuda.is_available()
    return m


def i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def same_bits(a, b):
    a, b = a.cpu().contiguous(), b.cpu().contiguous()
    return bool((a.view(torch.int16) == b.view(torch.int16)).all())


def draw(seed):
    r = random.Random(seed)
    D = r.choice([64, 96, 128, 192, 256])
    G = r.choice([g for g in (32, 64, 128) if D % g == 0])
    H = r.choice([1, 1, 2, 3])
    R = r.choice([1, 1, 2, 4, 5, 8, 17])
    batch = r.choice([1, 1, 2, 3, 5, 9])
    top = int(2 ** r.uniform(0, 10.5))
    lens = [r.choice([0, 1, top, r.randint(0, top)]) for _ in range(batch)]
    if r.random() < 0.3:
        new = [1] * batch
        lens = [max(1, n) for n in lens]
    else:
        most = r.choice([1, 3, 17, 70, 140])
        new = [min(n, r.randint(0, most)) for n in lens]
    return dict(D=D, G=G, H=H, R=R, lens=lens, new=new, page=r.choice([16, 32, 128, 1024]),
                dt=r.choice([torch.float16, torch.bfloat16]), causal=r.random() < 0.7,
                window=r.choice([0, 0, r.randint(1, top + 1)]), scale=r.choice([None, 0.02, 0.5]),
                max_kv=r.choice([None, 0, top, 50000]), strided=r.random() < 0.5, cuts=r.randint(1, 4), r=r)


@pytest.mark.parametrize("seed", range(120))
def test_random_problem(wq, seed):
    c = draw(seed)
    print({k: v for k, v in c.items() if k != "r"}, flush=True)
    D, H, Hq, dt, r = c["D"], c["H"], c["H"] * c["R"], c["dt"], c["r"]
    lens, new = c["lens"], c["new"]
    P = _kv.Problem(lens, new, H, D, c["G"], c["page"], dt, seed)
    cache, table = P.empty(wq), P.table.cuda()
    # written in up to four pieces, cut at random
    at = [0] * len(lens)
    for i in range(c["cuts"]):
        to = [n if i == c["cuts"] - 1 else r.randint(a, n) for a, n in zip(at, lens)]
        counts = [t - a for a, t in zip(at, to)]
        k = torch.cat([x[a:t] for x, a, t in zip(P.K, at, to)])
        v = torch.cat([x[a:t] for x, a, t in zip(P.V, at, to)])
        if c["strided"]:
            both = torch.zeros(k.shape[0], 2 * H + 1, D, dtype=dt, device="cuda")
            both[:, :H], both[:, H + 1:] = k.cuda(), v.cuda()
            k, v = both[:, :H], both[:, H + 1:]
        wq.wq_kv_write(k.cuda(), v.cuda(), cache, table, i32(to), cu_q=P.cu(counts).cuda())
        at = to
    k, v = wq.wq_kv_read(cache, table, i32(lens), sum(lens), cu_q=P.cu(lens).cuda())
    assert same_bits(k, _kv.stored(torch.cat(P.K), c["G"])) and same_bits(v, _kv.stored(torch.cat(P.V), c["G"]))
    T = sum(new)
    q = P.queries(Hq)
    qd = q.cuda()
    if c["strided"]:
        wide = torch.full((T, Hq + 2, D), 3.0, dtype=dt, device="cuda")
        wide[:, 1:Hq + 1] = qd
        qd = wide[:, 1:Hq + 1]
    uniform = len(set(new)) == 1 and r.random() < 0.5
    scale = c["scale"] or D ** -0.5
    out = wq.wq_kv_attention(qd, cache, table, i32(lens), cu_q=None if uniform else P.cu(new).cuda(), scale=c["scale"],
                             causal=c["causal"], window=c["window"], max_kv_len=c["max_kv"])
    want, bound = P.reference(q, scale, c["causal"], c["window"])
    err = (out.cpu().double() - want).abs()
    assert bool((err <= bound).all()), float((err / bound).max())
    again = wq.wq_kv_attention(qd, cache, table, i32(lens), cu_q=None if uniform else P.cu(new).cuda(),
                               scale=c["scale"], causal=c["causal"], window=c["window"], max_kv_len=c["max_kv"])
    assert same_bits(out, again)

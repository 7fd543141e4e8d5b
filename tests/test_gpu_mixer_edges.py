"""GPU: the token mixers at what a norm over a whole result does not see: values that are not finite, results as a
whole against their correctly rounded values, tokens and heads one by one, calls from several threads and streams."""

import threading

import numpy as np
import pytest
import torch

import mixer_reference as ref
from test_gpu_mixers import DT, cache_of, delta_inputs, fmoe, near, paged, state_bound  # noqa: F401 (fmoe: a fixture)

pytestmark = pytest.mark.gpu


def flips(got, want, dtype, b, what):
    """`got` against `want` (binary64) rounded to `dtype`, 2-norms over the last axis and all before it.

    A value that is off by d before its rounding lands on the neighbour of the right result with probability d / step,
    and is then off by a step: the square of the difference is the sum of step * |d| on average, at most |step| |d| in
    2-norms. With |d| <= b |want| and steps of eps |want| at most that is eps b |want|^2; twice the root for the spread."""
    rounded = torch.from_numpy(want).to(dtype).double().numpy()
    off = np.linalg.norm(ref.f64(got) - rounded) / np.linalg.norm(want)
    bound = 2 * (torch.finfo(dtype).eps * b) ** 0.5
    assert off <= bound, f"{what}: {off:.3e} > {bound:.3e}"


# ------------------------------------------------------------------------------------------------ delta rule
def delta_parts(q, k, v, g, beta, S, scale, eps=1e-6):
    """One sequence as ref.delta, l2norm on, and for each token what its result is summed from: out, state, u,
    |q~|^T |S| of the state before the token's chunk as far as it has not decayed, and sum |q~ k~| |u| over the tokens
    of the chunk up to it (both times scale)."""
    t, hv, dv = v.shape
    rep = hv // k.shape[1]
    q, k = (np.repeat(x / np.sqrt((x * x).sum(-1, keepdims=True) + eps), rep, 1) for x in (q, k))
    S, out, us = S.copy(), np.zeros((t, hv, dv)), np.zeros((t, hv, dv))
    old, new = np.zeros((t, hv, dv)), np.zeros((t, hv, dv))
    for i in range(t):
        if i % 64 == 0:
            before, since = np.abs(S), np.zeros((hv, 0))
        e = np.exp(g[i])
        before, since = before * e[:, None, None], np.concatenate([since * e[:, None], np.ones((hv, 1))], 1)
        S = S * e[:, None, None]
        us[i] = beta[i][:, None] * (v[i] - np.einsum("hkv,hk->hv", S, k[i]))
        S = S + k[i][:, :, None] * us[i][:, None, :]
        out[i] = scale * np.einsum("hkv,hk->hv", S, q[i])
        old[i] = scale * np.einsum("hkv,hk->hv", before, np.abs(q[i]))
        c = i - i % 64
        meet = np.abs(np.einsum("hk,jhk->hj", q[i], k[c:i + 1])) * since
        new[i] = scale * np.einsum("hj,jhv->hv", meet, np.abs(us[c:i + 1]))
    return out, S, us, old, new


def check_tokens(got, got_state, x, lens, dtype):
    """Every token and head by itself. Terms: the result's rounding; M and U in binary16 (2^-12 each) for a bfloat16
    result, in 22 bits (2^-21 for both) for a binary16 one; the state and the sums, as state_bound; and the limit that
    fmoe.h gives: 2^-39 of the largest that a column meets within the chunk, 64 of them in a sum, in each of the right-
    hand side, U, and T; and 2^-65 in every entry of the state, before every chunk. That is up to sqrt(dk) 2^-65 in k~ S,
    so in each token's right-hand side, and a token adds as much (times beta <= 1 and |k~| <= 1) to the error of its
    column of the state, which the rule contracts: sqrt(dk) 2^-65 a token so far, times sqrt(dv) for all columns."""
    q, k, v, g, beta = (ref.f64(t) for t in x[:5])
    state0, slots, cu = ref.f64(x[5]), x[6].tolist(), x[7].tolist()
    dk = k.shape[-1]
    got, got_state, scale = ref.f64(got), ref.f64(got_state), dk ** -0.5
    eps, operand = torch.finfo(dtype).eps / 2, 2.0 ** (-11 if dtype == torch.bfloat16 else -21)
    for i, n in enumerate(lens):
        b = cu[i]
        out, S, us, old, new = delta_parts(q[b:b + n], k[b:b + n], v[b:b + n], g[b:b + n], beta[b:b + n], state0[slots[i]], scale)
        for t in range(n):
            c = t - t % 64
            top = np.maximum(np.abs(us[c:c + 64]), np.abs(v[b + c:b + n][:64])).max(0)  # [heads, columns]
            bound = (eps * np.linalg.norm(out[t], axis=-1) + operand * np.linalg.norm(new[t], axis=-1)
                     + 4 * state_bound(dk) * (np.linalg.norm(old[t], axis=-1) + np.linalg.norm(new[t], axis=-1))
                     + scale * (3 * 64 * 2.0 ** -39 * np.linalg.norm(top, axis=-1) + (t + 2) * 2.0 ** -65 * (dk * v.shape[-1]) ** 0.5))
            off = np.linalg.norm(got[b + t] - out[t], axis=-1)
            assert (off <= bound).all(), (i, t, (off / bound).max())
        top = np.abs(us[n - 1 - (n - 1) % 64:]).max(0)
        bound = (2 * state_bound(dk) * np.linalg.norm(S, axis=(1, 2)) + 3 * 64 * 2.0 ** -39 * np.linalg.norm(top, axis=-1)
                 + (n + 1) * 2.0 ** -65 * (dk * v.shape[-1]) ** 0.5)
        off = np.linalg.norm(got_state[slots[i]] - S, axis=(1, 2))
        assert (off <= bound).all(), (i, "state", (off / bound).max())


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("large", [False, True])
def test_delta_chunk_extreme_values_by_token(fmoe, dtype, large):
    """Zero keys and queries, huge and tiny keys, beta 0 and 1, each token by itself; values 2^20 times the others, in
    the same chunk (bfloat16)."""
    lens = [100]
    x = list(delta_inputs(lens, 2, 2, 64, 64, DT[dtype], 5))
    q, k, v = (t.clone() for t in x[:3])
    far = 2.0 ** 40 if dtype == "bf16" else 2.0 ** 10
    k[3], k[10], k[11], q[7] = 0, k[10] * far, k[11] / far, 0
    if large:
        v[30:40] *= 2.0 ** (20 if dtype == "bf16" else 10)
    x[:3] = q, k, v
    x[4][::5], x[4][1::5] = 0, 1
    state = x[5].clone()
    out = fmoe.delta_chunk(*x[:5], state, x[7], 100, slots=x[6])
    assert fmoe.sync_status() == 0
    check_tokens(out, state, x, lens, DT[dtype])


@pytest.mark.parametrize("decay", [0.0, 0.02, 3.0])
def test_delta_chunk_stretches_by_token(fmoe, decay):
    """Values whose size falls and rises by 2^12 or 2^24; the sequences end in a stretch of small ones."""
    lens = [700, 520]
    x = list(delta_inputs(lens, 2, 2, 128, 64, torch.bfloat16, 22, decay=decay))
    v = x[2].clone()
    for i, size in enumerate((0, 12, -12, 12, -12)):  # 140 tokens each
        v[140 * i:140 * (i + 1)] *= 2.0 ** size
    for i, size in enumerate((12, 0, -12, -12)):  # 130 each
        v[700 + 130 * i:700 + 130 * (i + 1)] *= 2.0 ** size
    x[2] = v
    state = x[5].clone()
    out = fmoe.delta_chunk(*x[:5], state, x[7], 700, slots=x[6])
    assert fmoe.sync_status() == 0
    check_tokens(out, state, x, lens, torch.bfloat16)


@pytest.mark.parametrize("size", [2.0 ** -45, 2.0 ** 60])
def test_delta_chunk_of_any_size(fmoe, size):
    """Values and states far from 1 in size."""
    lens = [200, 65]
    x = list(delta_inputs(lens, 2, 2, 128, 64, torch.bfloat16, 23))
    x[2], x[5] = x[2] * size, x[5] * size
    state = x[5].clone()
    out = fmoe.delta_chunk(*x[:5], state, x[7], 200, slots=x[6])
    assert fmoe.sync_status() == 0
    check_tokens(out, state, x, lens, torch.bfloat16)


@pytest.mark.parametrize("lens,dk,dv", [([64], 64, 64), ([300, 77], 128, 128), ([1000], 64, 128)], ids=str)
def test_delta_chunk_binary16_results(fmoe, lens, dk, dv):
    """Binary16 results are those of binary32 arithmetic, rounded once."""
    x = delta_inputs(lens, 2, 4, dk, dv, torch.float16, 30)
    state = x[5].clone()
    out = fmoe.delta_chunk(*x[:5], state, x[7], max(lens), slots=x[6])
    assert fmoe.sync_status() == 0
    a = [ref.f64(t) for t in x[:6]]
    want = []
    for i, n in enumerate(lens):
        b = int(x[7][i])
        want.append(ref.delta(*(t[b:b + n] for t in a[:5]), a[5][int(x[6][i])], dk ** -0.5, True, 1e-6)[0])
    flips(out, np.concatenate(want), torch.float16, state_bound(dk), "out")


@pytest.mark.parametrize("dtype,most", [("bf16", 70), ("fp32", 70), ("bf16", 0)])
def test_delta_chunk_padding_layers_and_broadcast(fmoe, dtype, most):
    """A padded sequence and one of a bad slot among others, states that are one layer's slice of a larger array, gates that
    are slices, a key shared by all heads and tokens: what contiguous copies give, and nothing else written."""
    lens, hv, d = [70, 30, 64, 9], 4, 64
    x = list(delta_inputs(lens, 2, hv, d, d, DT[dtype], 60))
    t = sum(lens)
    layers = 0.3 * torch.randn(6, 3, hv, d, d, device="cuda", generator=torch.Generator(device="cuda").manual_seed(61))
    gates = torch.randn(t, 3 * hv, device="cuda", generator=torch.Generator(device="cuda").manual_seed(62))
    gates[:, :hv] = -gates[:, :hv].abs()
    gates[:, hv:2 * hv].sigmoid_()
    k = x[1][:1, :1].expand(t, 2, d)
    slots = torch.tensor([4, -1, 0, 6], dtype=torch.int32, device="cuda")
    before, out = layers.clone(), torch.full((t, hv, d), 7.0, dtype=DT[dtype], device="cuda")
    fmoe.delta_chunk(x[0], k, x[2], gates[:, :hv], gates[:, hv:2 * hv], layers[:, 1], x[7], most, slots=slots, out=out)
    assert fmoe.sync_status() == fmoe.FMOE_ERR_INDEX and "slot" in fmoe.last_error()
    state = before[:, 1].contiguous()
    good = torch.tensor([4, 5, 0, 2], dtype=torch.int32, device="cuda")
    want = fmoe.delta_chunk(x[0].contiguous(), k.contiguous(), x[2].contiguous(), gates[:, :hv].contiguous(),
                            gates[:, hv:2 * hv].contiguous(), state, x[7], most, slots=good)
    assert fmoe.sync_status() == 0
    for i, (a, b) in enumerate(zip(x[7].tolist(), x[7].tolist()[1:])):
        assert torch.equal(out[a:b], want[a:b]) if i in (0, 2) else (out[a:b] == 7).all()
    for i in range(6):
        assert torch.equal(layers[i, 1], state[i] if i in (4, 0) else before[i, 1])
    assert torch.equal(layers[:, 0], before[:, 0]) and torch.equal(layers[:, 2], before[:, 2])


@pytest.mark.parametrize("dtype,most", [("bf16", 70), ("bf16", 0)])
def test_delta_offsets_beyond_32_bits(fmoe, dtype, most):
    """States and rows whose elements lie beyond 2^31."""
    hv, d, step, t = 64, 128, 1 << 25, 70
    wide = torch.empty(3, t * step // 2, dtype=torch.bfloat16, device="cuda")  # 3 x 2.3 GB: rows step / 2 apart, q, k, v
    x = list(delta_inputs([t], 2, hv, d, d, torch.bfloat16, 63))
    far = [torch.as_strided(wide.view(-1), (t, a.shape[1], d), (step * 3 // 2, d, 1), i * 16384) for i, a in enumerate(x[:3])]
    for a, b in zip(far, x[:3]):
        a.copy_(b)
    assert (t - 1) * step * 3 // 2 > 2 ** 31
    state = torch.empty(2060, hv, d, d, device="cuda")  # 8.6 GB
    slots = torch.tensor([2059], dtype=torch.int32, device="cuda")
    state[2059] = x[5][0]
    few = x[5][:1].clone()
    want = fmoe.delta_chunk(*x[:5], few, x[7], most)
    out = torch.as_strided(wide.view(-1), (t, hv, d), (step * 3 // 2, d, 1), 3 * 16384)
    fmoe.delta_chunk(*far, *x[3:5], state, x[7], most, slots=slots, out=out)
    assert fmoe.sync_status() == 0
    assert torch.equal(out, want) and torch.equal(state[2059], few[0])


NAN, INF = float("nan"), float("inf")


ODD = [("k", NAN), ("k", -INF), ("q", NAN), ("q", INF), ("v", NAN), ("v", INF), ("v", -INF), ("g", NAN), ("g", INF),
       ("beta", NAN), ("beta", INF), ("state", NAN), ("state", -INF)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("what,value", ODD, ids=str)
@pytest.mark.parametrize("l2norm", [True, False])
def test_delta_chunk_not_finite(fmoe, dtype, what, value, l2norm):
    """What is not finite reaches its own token and those behind it (of its column, where it is a value or an entry of
    the state; its token alone, where it is a query), as in the recurrent form, and nothing else."""
    lens, dk, dv = [150, 30, 64], 64, 128
    for at in (0, 20, 63, 64, 149):
        x = list(delta_inputs(lens, 2, 4, dk, dv, DT[dtype], 40))
        x = [t.clone() for t in x]
        if not l2norm:
            x[0], x[1] = x[0] * 0.09375, x[1] * 0.09375
        x[1][:, :, 7] = 1 / 16  # no key component that is zero in these columns
        if what == "state":
            x[5][x[6][0], 1, 5, 9] = value
        elif what in "gbeta":
            x["g beta".split().index(what) + 3][at, 1] = value
        else:
            i = "qkv".index(what)
            x[i][at, 1, 7] = value
            if what == "q":  # and one in every 16 tokens of the last sequence, and of a short chunk
                x[0][180::16, 0, 3] = value
                x[0][155, 0, 3] = value
        want_state, state = x[5].clone(), x[5].clone()
        want = fmoe.delta_chunk(*x[:5], want_state, x[7], 0, slots=x[6], l2norm=l2norm)
        out = fmoe.delta_chunk(*x[:5], state, x[7], 150, slots=x[6], l2norm=l2norm)
        assert fmoe.sync_status() == 0
        ok, ok_state = torch.isfinite(want), torch.isfinite(want_state)
        assert not ok.all()
        assert torch.equal(torch.isfinite(out), ok), (at, "out")
        assert torch.equal(torch.isfinite(state), ok_state), (at, "state")
        # two forms, each within the bound, and two roundings
        d = DT[dtype]
        for t in range(0, sum(lens), 10):
            near(torch.where(ok[t:t + 10], out[t:t + 10], 0), ref.f64(torch.where(ok[t:t + 10], want[t:t + 10], 0)), d,
                 torch.finfo(d).eps / 2 + 2 ** -11 + 2 * state_bound(dk), f"{at}: out from {t}")
        near(torch.where(ok_state, state, 0), ref.f64(torch.where(ok_state, want_state, 0)), torch.float32,
             2 * state_bound(dk), f"{at}: state")


@pytest.mark.parametrize("dtype", list(DT))
def test_delta_rows_of_zeros_without_eps(fmoe, dtype):
    """Keys and queries of zeros stay zeros where they are divided by a norm of zero, in every form."""
    lens, dk, dv = [40, 17], 64, 64
    x = [t.clone() for t in delta_inputs(lens, 2, 2, dk, dv, DT[dtype], 44)]
    x[1][5], x[0][9], x[1][45, 1] = 0, 0, 0
    a = [ref.f64(t) for t in x[:6]]
    a[0], a[1] = (t / np.maximum(np.linalg.norm(t, axis=-1, keepdims=True), 1e-30) for t in a[:2])
    for most in (0, 40):
        state = x[5].clone()
        out = fmoe.delta_chunk(*x[:5], state, x[7], most, slots=x[6], eps=0.0)
        assert fmoe.sync_status() == 0
        for i, n in enumerate(lens):
            b, slot = int(x[7][i]), int(x[6][i])
            o, S = ref.delta(*(t[b:b + n] for t in a[:5]), a[5][slot], dk ** -0.5, False, 0.0)
            near(out[b:b + n], o, DT[dtype], 2 ** -11 * (dtype == "bf16") + state_bound(dk), (most, "out"))
            near(state[slot], S, torch.float32, state_bound(dk), (most, "state"))
    one = [t[5:6].contiguous() for t in x[:5]]
    state = x[5].clone()
    out = fmoe.delta_step(*one, state, slots=x[6][:1], eps=0.0)
    o, S = ref.delta(*(t[5:6] for t in a[:5]), a[5][int(x[6][0])], dk ** -0.5, False, 0.0)
    near(out, o, DT[dtype], state_bound(dk), "step")
    near(state[x[6][0]], S, torch.float32, state_bound(dk), "step's state")


# ------------------------------------------------------------------------------------------------ the cache
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("d", [64, 128, 256])
def test_append_not_finite(fmoe, dtype, d):
    """64 columns with a NaN or an infinity among them are read back as no numbers, all of them, wherever it stands;
    the others are as without it."""
    ps, n = 16, 64
    gen = torch.Generator(device="cuda").manual_seed(d)
    x = torch.randn(n, 2, d, generator=gen, device="cuda").to(DT[dtype])
    odd = x.clone()
    for t in range(n):
        odd[t, t % 2, (t * 5) % d] = (NAN, INF, -INF)[t % 3]
    P, S = torch.arange(n, dtype=torch.int32, device="cuda"), torch.zeros(n, dtype=torch.int32, device="cuda")
    table = torch.arange(n // ps, dtype=torch.int32, device="cuda")[None]
    held = []
    for rows in (x, odd):
        pages = fmoe.kv_pages(n // ps, 2, d, ps)
        fmoe.kv_append(rows, rows, P, pages, table, torch.zeros(0, device="cuda"), seq=S)
        held.append(fmoe.kv_read(pages, table, P, d, seq=S, dtype=torch.float32))
    assert fmoe.sync_status() == 0
    hit = ~torch.isfinite(odd.float()).view(n, 2, d // 64, 64).all(-1, keepdim=True).expand(n, 2, d // 64, 64).reshape(n, 2, d)
    for clean, got in zip(*held):
        assert not torch.isfinite(got[hit]).any()
        assert torch.equal(got[~hit], clean[~hit])


def test_cache_beyond_32_bits(fmoe):
    """Pages that lie beyond 2^32 bytes, through a slice of a wider table: as in a small cache."""
    d, ps, hkv, n = 256, 1024, 8, 1500
    gen = torch.Generator(device="cuda").manual_seed(64)
    kv = torch.randn(n, 2 * hkv, d, generator=gen, device="cuda").to(torch.bfloat16)
    q = torch.randn(1, 16, d, generator=gen, device="cuda").to(torch.bfloat16)
    P, S = torch.arange(n, dtype=torch.int32, device="cuda"), torch.zeros(n, dtype=torch.int32, device="cuda")
    L = torch.tensor([n], dtype=torch.int32, device="cuda")
    got = []
    for pages, ids in ((fmoe.kv_pages(2, hkv, d, ps), [1, 0]),
                       (torch.empty(2000, hkv, fmoe.kv_block_bytes(ps, d), dtype=torch.uint8, device="cuda"), [1999, 1960])):
        wide = torch.full((1, 9), -1, dtype=torch.int32, device="cuda")
        wide[0, 4:6] = torch.tensor(ids, dtype=torch.int32)
        table = wide[:, 4:6]
        fmoe.kv_append(kv[:, :hkv], kv[:, hkv:], P, pages, table, torch.zeros(0, device="cuda"), seq=S)
        got.append([*fmoe.kv_read(pages, table, P, d, seq=S), fmoe.attn_q4(q, pages, table, L, n)])
    assert pages.stride(0) * 1960 > 2 ** 32 and fmoe.sync_status() == 0
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_append_padding_leaves_queries(fmoe):
    d, ps = 64, 16
    x = torch.randn(4, 4, d, device="cuda", generator=torch.Generator(device="cuda").manual_seed(65))
    pages, table = fmoe.kv_pages(4, 1, d, ps), torch.arange(4, dtype=torch.int32, device="cuda")[:, None]
    P = torch.tensor([3, -1, 0, -7], dtype=torch.int32, device="cuda")
    out = torch.full((4, 2, d), 7.0, device="cuda")
    fmoe.kv_append(x[:, 2:3], x[:, 3:], P, pages, table, torch.ones(8, device="cuda"), q=x[:, :2], q_out=out)
    assert fmoe.sync_status() == 0
    assert (out[[1, 3]] == 7).all() and not (out[[0, 2]] == 7).any()
    assert not pages[[1, 3]].any() and pages[0].any() and pages[2].any()


# ------------------------------------------------------------------------------------------------ attention
def unpacked(pages, ps, d):
    """Pages of one kv head [pages, bytes] on the GPU -> keys, values [positions, d] in binary64."""
    codes = pages[:, :ps * d].reshape(-1, 2, ps, d // 2)
    q = torch.stack([codes & 15, codes >> 4], -1).reshape(-1, 2, ps, d // 64, 64).double()
    sb = pages[:, ps * d:].contiguous().view(torch.bfloat16).view(-1, 2, ps, d // 64, 2).double()
    x = (q * sb[..., :1] + sb[..., 1:]).reshape(-1, 2, ps, d)
    return x[:, 0].reshape(-1, d), x[:, 1].reshape(-1, d)


def like_weights(fmoe, dtype, n, requests, d, hq):  # noqa: F811
    """Positions of like weight whose values average out: a result of about |v| / sqrt(n) from terms of |v| / n. Several
    requests share their pages.

    Before the rounding to 16 bits a result is off, relative to itself, by: probabilities and their products with the
    scales, 2^-20 with the exponentials (terms of a few |v| / n, independent of one another); and the sums, whose terms
    come to 2 sqrt(n) results at most, all of one sign, rounded to nearest, 2^-24 with about sqrt(n) / 2 in a row of
    errors that average out: 2^-24 sqrt(n). For bfloat16 the products with the scales are rounded to binary16: 2^-12 of
    each of those terms, which come to twice the values."""
    ps, dt = 64, DT[dtype]
    pages, table = cache_of([n], 1, d, ps, 51, extra_pages=0)
    gen = torch.Generator(device="cuda").manual_seed(52)
    if requests > 1:
        order = torch.stack([torch.randperm(table.shape[1], generator=gen, device="cuda") for _ in range(requests)])
        table = table[0][order].contiguous()
    q = torch.randn(requests, hq, d, generator=gen, device="cuda").to(dt)
    L = torch.full((requests,), n, dtype=torch.int32, device="cuda")
    out = fmoe.attn_q4(q, pages, table, L, n, scale=0.3 / d)
    assert fmoe.sync_status() == 0
    k, v = unpacked(pages[:, 0][table[0].long()], ps, d)
    k, v = k[:n], v[:n]
    want = torch.cat([torch.softmax(q[i].double() @ k.T * (0.3 / d), -1) @ v for i in range(requests)]).cpu().numpy()
    got = out.view(-1, d)
    b = 2.0 ** -20 + 2.0 ** -24 * n ** 0.5
    if dtype == "fp32":
        off = np.linalg.norm(ref.f64(got) - want) / np.linalg.norm(want)
        assert off <= 4 * b, (off, 4 * b)
    else:
        flips(got, want, dt, b if dtype == "fp16" else 2.0 ** -11 + b, "out")


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("n,d,hq", [(64, 64, 8), (1000, 128, 16), (20000, 256, 32)], ids=str)
def test_attention_of_like_weights_as_a_whole(fmoe, dtype, n, d, hq):
    like_weights(fmoe, dtype, n, 1, d, hq)


@pytest.mark.parametrize("dtype", list(DT))
def test_attention_of_like_weights_in_long_shares(fmoe, dtype):
    """A warp has about 14000 positions one after another."""
    like_weights(fmoe, dtype, 131072, 256, 64, 8)


@pytest.mark.parametrize("scale", [0.0, 0.088, 2.0])
def test_attention_long_as_a_whole(fmoe, scale):
    """Binary32 results over many joined parts, head by head: logits of up to |x| are off by 2^-22 |x| and move every
    probability by as much, relative; the rest as above."""
    n, d, ps = 70001, 128, 64
    pages, table = cache_of([n], 2, d, ps, 9)
    q = torch.randn(1, 16, d, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2))
    out = fmoe.attn_q4(q, pages, table, torch.tensor([n], dtype=torch.int32, device="cuda"), n, scale=scale)
    assert fmoe.sync_status() == 0
    for h in range(2):
        k, v = unpacked(pages[:, h][table[0].long()], ps, d)
        x = q[0, 8 * h:8 * h + 8].double() @ k[:n].T * scale
        want = (torch.softmax(x, -1) @ v[:n]).cpu().numpy()
        top = float(x.abs().max())
        for r in range(8):
            off = np.linalg.norm(ref.f64(out[0, 8 * h + r]) - want[r]) / np.linalg.norm(want[r])
            assert off <= 4 * (2.0 ** -20 + 2.0 ** -24 * n ** 0.5 + 2.0 ** -22 * top), (h, r, off)


@pytest.mark.parametrize("dtype", list(DT))
def test_attention_small_scales_that_decide(fmoe, dtype):
    """Positions of large value scales and next to no weight beside positions of scales 2^-10 of theirs and all the
    weight. The product of weight and scale is held to 2^-12 of itself (bfloat16) or 2^-22, and to 2^-32 of the largest
    scale (fmoe.h), times codes of 16 at most; the rest as check_attn has it."""
    n, d, ps, dt, scale = 200, 64, 16, DT[dtype], 0.25
    pages, table = cache_of([n], 1, d, ps, 61)
    sb = pages[:, :, ps * d:].view(torch.bfloat16).view(-1, 1, 2, ps, 1, 2)
    for t in range(n):
        page, at = int(table[0, t // ps]), t % ps
        if t % 5 == 2:
            sb[page, 0, 0, at] = torch.tensor([0.0, -4.0], device="cuda").to(torch.bfloat16)  # -4 in all columns: a logit of -64
        else:
            sb[page, 0, 1, at] *= 2.0 ** -10
            sb[page, 0, 0, at] *= 2.0 ** -4
    q = (0.5 + torch.rand(1, 8, d, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))).to(dt)
    out = fmoe.attn_q4(q, pages, table, torch.tensor([n], dtype=torch.int32, device="cuda"), n, scale=scale)
    assert fmoe.sync_status() == 0
    mine = pages[:, 0][table[0].long()]
    k, v = (x[:n] for x in unpacked(mine, ps, d))
    sb = mine[:, ps * d:].contiguous().view(torch.bfloat16).view(-1, 2, ps, 2).double()
    sk, sv, zv = sb[:, 0, :, 0].reshape(-1)[:n], sb[:, 1, :, 0].reshape(-1)[:n], sb[:, 1, :, 1].reshape(-1)[:n]
    for r in range(8):
        x = scale * (k @ q[0, r].double())
        p = torch.softmax(x, -1)
        want = p @ v
        mass = scale * (k.abs() + 16 * sk[:, None]) @ q[0, r].double().abs()
        dx = 2 * (d + 8) * 2.0 ** -24 * float(mass.max()) + 2.0 ** -22 * (1 + float(x.abs().max()))
        codes = float(p @ (15 * sv + zv.abs()))
        bound = (torch.finfo(dt).eps / 2 * want.abs() + (2.0 ** (-12 if dtype == "bf16" else -21) + 2 * dx) * codes
                 + 2.0 ** -32 * n * 16 * float(sv.max()))
        off = (out[0, r].double() - want).abs()
        assert bool((off <= bound).all()), (r, float((off / bound).max()))


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("value", [NAN, INF, -INF])
def test_attention_values_not_finite(fmoe, dtype, value):
    """A value scale or bias that is not finite makes its 64 columns so, and no others."""
    n, d, ps = 100, 128, 16
    for part in (0, 1):
        pages, table = cache_of([n], 1, d, ps, 71)
        clean = pages.clone()
        sb = pages[:, :, ps * d:].view(torch.bfloat16).view(-1, 1, 2, ps, 2, 2)
        sb[int(table[0, 0]), 0, 1, 3, 0, part] = value
        q = torch.randn(1, 4, d, device="cuda", generator=torch.Generator(device="cuda").manual_seed(4)).to(DT[dtype])
        L = torch.tensor([n], dtype=torch.int32, device="cuda")
        out, want = fmoe.attn_q4(q, pages, table, L, n), fmoe.attn_q4(q, clean, table, L, n)
        assert fmoe.sync_status() == 0
        assert not torch.isfinite(out[..., :64]).any()
        assert torch.equal(out[..., 64:], want[..., 64:])


@pytest.mark.parametrize("most", [100, 9000])
def test_attention_counts_that_fall_back(fmoe, most):
    """A cu_q that falls, and lengths out of range of sequences without queries, are reported, whether thread blocks
    take whole items (short) or share all passes."""
    lens, d, ps = [100, 60, 90], 64, 16
    pages, table = cache_of([9000 if most > 100 else 100, 60, 90], 1, d, ps, 4)
    gen = torch.Generator(device="cuda").manual_seed(5)
    q = torch.randn(8, 2, d, generator=gen, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")

    def status(cu, lengths):
        out = fmoe.attn_q4(q, pages, table, torch.tensor(lengths, **i32), most, cu_q=torch.tensor(cu, **i32), max_q=5)
        return out, fmoe.sync_status()
    good, code = status([0, 3, 5, 8], lens)
    assert code == 0
    got, code = status([0, 3, 3, 8], lens)
    assert code == 0 and torch.equal(got[:3], good[:3])
    for cu, lengths in (([0, 5, 3, 8], lens), ([0, 3, 3, 8], [100, -5, 90]), ([0, 3, 3, 8], [100, 10 ** 6, 90]),
                        ([0, 8, 8, 2], lens)):
        _, code = status(cu, lengths)
        assert code == fmoe.FMOE_ERR_INDEX and "length" in fmoe.last_error(), (cu, lengths)
    assert fmoe.sync_status() == 0


@pytest.mark.parametrize("most", [100, 9000])
def test_attention_counts_of_any_numbers(fmoe, most):
    """Whatever stands in cu_q: rows outside 0 .. n_tokens are not touched, and it is reported."""
    lens, d, ps = [100, 60], 64, 16
    pages, table = cache_of([most, 60], 1, d, ps, 4)
    wide = torch.randn(72, 2, d, device="cuda", generator=torch.Generator(device="cuda").manual_seed(5))
    out = torch.full_like(wide, 7.0)
    L = torch.tensor(lens, dtype=torch.int32, device="cuda")
    low, high = -2 ** 31, 2 ** 31 - 1
    for cu in ([0, 5, low], [5, low, 8], [0, 5, -3], [low, 5, 8], [0, high, 8], [8, high, low], [low, high, 8], [7, 8, high]):
        fmoe.attn_q4(wide[32:40], pages, table, L, most, cu_q=torch.tensor(cu, dtype=torch.int32, device="cuda"), max_q=32, out=out[32:40])
        assert fmoe.sync_status() == fmoe.FMOE_ERR_INDEX and "length" in fmoe.last_error(), cu
        assert (out[:32] == 7).all() and (out[40:] == 7).all(), cu


def test_attention_of_2_31_passes(fmoe):
    """More than 2^31 passes: a table that names one page again and again, and a bound of the queries that gives 65520
    blocks of rows, all empty but one. The result is that of the one page, but for sums of up to 2^17 terms in a row:
    2^-25 each of up to four results."""
    d, ps, times = 64, 1024, 1026
    pages, one = cache_of([ps], 1, d, ps, 81, extra_pages=0)
    q = torch.randn(1, 2, d, device="cuda", generator=torch.Generator(device="cuda").manual_seed(6))
    table = one.expand(1, times).contiguous()
    cu = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    n, most = ps * times, 65520 * 128 // 2  # 128 rows of two heads a block
    assert n // 32 * 65520 > 2 ** 31
    out = fmoe.attn_q4(q, pages, table, torch.tensor([n], dtype=torch.int32, device="cuda"), n, cu_q=cu, max_q=most, scale=0.2)
    assert fmoe.sync_status() == 0
    k, v = unpacked(pages[:, 0], ps, d)
    want = (torch.softmax(q[0].double() @ k.T * 0.2, -1) @ v).cpu().numpy()
    off = np.linalg.norm(ref.f64(out[0]) - want) / np.linalg.norm(want)
    assert off <= 4 * 2.0 ** -8, off


# ------------------------------------------------------------------------------------------------ as they are used
def test_attention_from_two_threads(fmoe):
    """Two host threads, each with its stream, whose calls run one kernel with different amounts of shared memory: none
    is refused, and the results are those of one thread."""
    d, ps, lens = 256, 64, [200, 130]
    pages, table = cache_of(lens, 1, d, ps, 91)
    L = torch.tensor(lens, dtype=torch.int32, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(7)
    cache, calls = fmoe._cache(pages.get_device(), pages, table, d), []
    for m in (1, 2):  # 16 rows of two tiles: one warp's, two warps'
        q = torch.randn(2 * m, 16, d, generator=gen, device="cuda").to(torch.bfloat16)
        cu = torch.tensor([0, m, 2 * m], dtype=torch.int32, device="cuda")
        want = fmoe.attn_q4(q, pages, table, L, 200, cu_q=cu, max_q=m)
        out = torch.zeros_like(want)
        desc = fmoe.AttnDesc(16, fmoe.FMOE_BF16, 2 * m, m, 200, d ** -0.5, q.data_ptr(), 16 * d, d, cu.data_ptr(),
                             L.data_ptr(), out.data_ptr(), 16 * d, d)
        calls.append((desc, want, out, q, cu, torch.cuda.Stream()))
    torch.cuda.synchronize()
    attn, codes = fmoe.lib().fmoe_attn_q4, [set(), set()]

    def work(i):
        desc, stream = calls[i][0], calls[i][-1].cuda_stream
        for _ in range(20000):
            codes[i].add(attn(cache, desc, stream))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert codes == [{0}, {0}] and fmoe.sync_status() == 0, codes
    torch.cuda.synchronize()
    for _, want, out, *_ in calls:
        assert torch.equal(out, want)


def test_results_on_another_stream(fmoe):
    """A result that a call makes for itself on the stream it is given is not memory that the current stream still
    writes."""
    n, hv, d, ps = 64, 8, 64, 16
    x = delta_inputs([1] * n, 4, hv, d, d, torch.bfloat16, 3)
    pages, table = cache_of([20] * n, 4, d, ps, 8)
    L = torch.full((n,), 20, dtype=torch.int32, device="cuda")
    q = torch.randn(n, hv, d, device="cuda").to(torch.bfloat16)
    P, inv = torch.zeros(n, dtype=torch.int32, device="cuda"), torch.ones(8, device="cuda")
    cu = torch.arange(n + 1, dtype=torch.int32, device="cuda")
    k = torch.randn(n, 4, d, device="cuda").to(torch.bfloat16)
    state = x[5].clone()
    calls = [lambda s: fmoe.delta_step(*x[:5], state, slots=x[6], stream=s),
             lambda s: fmoe.delta_chunk(*x[:5], state, cu, 1, slots=x[6], stream=s),
             lambda s: fmoe.attn_q4(q, pages, table, L, 20, stream=s),
             lambda s: fmoe.kv_append(k, k, P, pages, table, inv, q=q, stream=s)]
    st = torch.cuda.Stream()
    for call in calls:
        state.copy_(x[5])
        want = call(None).clone()
        state.copy_(x[5])
        out = call(0)  # the default stream by its handle, here the current one
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        for s in (st, st.cuda_stream):
            state.copy_(x[5])
            torch.cuda.synchronize()
            held = torch.empty(n, hv, d, dtype=torch.bfloat16, device="cuda")
            at = held.data_ptr()
            torch.cuda._sleep(20_000_000)  # about 10 ms, and then a write, of which the allocator knows by the stream's order
            held.fill_(7)
            del held
            out = call(s)
            assert out.data_ptr() != at
            torch.cuda.synchronize()
            assert torch.equal(out, want)
    assert fmoe.sync_status() == 0


def test_prompts_captured_and_replayed(fmoe):
    """A prompt's calls in one graph, replayed on other inputs, lengths, positions and slots: what eager calls give."""
    lens, others, d, ps = [70, 33], [21, 82], 128, 16
    sets = []
    for seed, ls in ((1, lens), (2, others)):
        x = delta_inputs(ls, 2, 4, d, d, torch.bfloat16, seed)
        gen = torch.Generator(device="cuda").manual_seed(seed)
        kv = torch.randn(103, 12, d, generator=gen, device="cuda").to(torch.bfloat16)
        pos = torch.cat([torch.arange(n) for n in ls]).to("cuda", torch.int32)
        seq = torch.repeat_interleave(torch.arange(2), torch.tensor(ls)).to("cuda", torch.int32)
        sets.append([*(t.contiguous() for t in x), kv, pos, seq, torch.tensor(ls, dtype=torch.int32, device="cuda")])
    inv = torch.rand(32, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))
    table, n_pages = paged(2, 96, ps, 5)

    def calls(q, k, v, g, beta, state, slots, cu, kv, pos, seq, L, pages):
        o = fmoe.delta_chunk(q, k, v, g, beta, state, cu, 96, slots=slots)
        turned = fmoe.kv_append(kv[:, 8:10], kv[:, 10:], pos, pages, table, inv, seq=seq, q=kv[:, :8])
        a = fmoe.attn_q4(turned, pages, table, L, 96, cu_q=cu, max_q=96)
        return [o, turned, a, *fmoe.kv_read(pages, table, pos, d, seq=seq), state, pages]
    want = [[t.clone() for t in calls(*(t.clone() for t in s), fmoe.kv_pages(n_pages, 2, d, ps))] for s in sets]
    held, pages = [t.clone() for t in sets[0]], fmoe.kv_pages(n_pages, 2, d, ps)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = calls(*held, pages)
    for i in (1, 0, 1):
        for a, b in zip(held, sets[i]):
            a.copy_(b)
        pages.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want[i]):
            assert torch.equal(a, b)
    assert fmoe.sync_status() == 0

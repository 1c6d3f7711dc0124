"""The 4-bit key/value cache on the GPU against the fp64 oracle.

Storing and reading back are exact: codes, scale bits and values equal the
oracle's.

Attention's tolerance, per output element.  The kernels round the levels (or
level times scale) to fp16, at most 2^-11 relative each and at most twice,
which moves a score by at most d = 2^-10 max_j sum_k |scale q_k k_jk| and so a
softmax weight by at most exp(2 d) - 1; the weights and the values' levels are
rounded to fp16 once and twice (3 * 2^-11 relative), and the output once to
bf16 (half an ulp, at most 2^-8 relative).  With the weighted mean of |v| as
the unit of all but the last:
    |out - ref| <= 2^-8 |ref| + (exp(2 d) - 1 + 3 * 2^-11) sum_j p_j |v_j|
plus fp32 sums' 2^-20 of the same unit, and |lse - ref| <= d + 2^-20 (1 + |ref|).
The whole output also meets the layer's relative Frobenius bound, 5e-3.
"""

import numpy as np
import pytest

from gpu_util import FRO_TOL, bf16_f64, dev_bf16, dev_f32, host, host_bf16_bits
from oracle import kv_oracle

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - the GPU suite needs an MI355X
    pytest.skip("no GPU", allow_module_level=True)

import bit_nf4_quantized_quant_amd as qa  # noqa: E402


def ints(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def tensors(cache):
    """Host copies (k_codes, k_scale bits, v_codes, v_scale bits)."""
    return (host(cache.k_codes), host_bf16_bits(cache.k_scales), host(cache.v_codes), host_bf16_bits(cache.v_scales))


# ------------------------------------------------------------------ store and read back

def awkward(rng, T, H, D):
    """fp32 tokens with the runs where the storing rule can go wrong."""
    x = rng.normal(0, 1, (T, H, D)).astype(np.float32)
    runs = x.reshape(-1, 64)
    for i, kind in enumerate(range(runs.shape[0])):
        kind = i % 12
        if kind == 1:
            runs[i] = 0
        elif kind == 2:
            runs[i] *= np.float32(1e-39)                      # subnormal magnitudes: stored as zero
        elif kind == 3:
            runs[i] *= np.float32(1e37)
            runs[i, 5] = np.finfo(np.float32).max             # the scale stops at the largest bf16
        elif kind == 4:
            runs[i] = 0
            runs[i, 63] = -3.0
        elif kind == 5:                                       # quotients at and next to the midpoints
            lv = kv_oracle.levels_f32(i // 12 % 3).astype(np.float64)
            mid = ((lv[1:] + lv[:-1]) / 2).astype(np.float32)
            m = np.concatenate([mid, np.nextafter(mid, np.float32(2)), np.nextafter(mid, np.float32(-2))])
            runs[i] = 0
            runs[i, :45] = m
            runs[i, 63] = 1.0
        elif kind == 6:
            runs[i] = np.float32(2.0 ** -126) * np.sign(runs[i])
        elif kind == 7:
            runs[i] = np.float32(1.00390625) * np.sign(runs[i])   # bf16 rounds the scale down
    return x


@pytest.mark.parametrize("table", [0, 1, 2])
@pytest.mark.parametrize("T,H,D,page,f32", [(1, 1, 64, 16, True), (37, 3, 128, 16, True), (131, 5, 256, 48, True),
                                            (67, 2, 64, 32, False), (129, 8, 128, 64, False), (5, 7, 256, 16, False)])
def test_store_and_read_back_are_exact(table, T, H, D, page, f32):
    rng = np.random.default_rng(7000 + T + 1000 * table + D)
    k, v = awkward(rng, T, H, D), awkward(rng, T, H, D)[::-1].copy()
    if not f32:
        k, v = (kv_oracle.bits_f64(np.minimum(kv_oracle.bf16_bits(np.abs(x)), 0x7F7F)).astype(np.float32) * np.sign(x)
                for x in (k, v))
    pages = -(-T // page) + 3
    slots = rng.permutation(pages * page)[:T].astype(np.int32)
    slots[T // 2::5] = np.where(np.arange(len(slots[T // 2::5])) % 2, -1, pages * page)[:len(slots[T // 2::5])]
    keep = (slots >= 0) & (slots < pages * page)
    cache = qa.kv_cache(pages, page, H, D, table=table)
    if f32:
        qa.kv_write(dev_f32(k), dev_f32(v), cache, ints(slots))
    else:                                                     # slices of a fused projection's output
        both = torch.cat([torch.zeros(T, H, D), torch.from_numpy(k), torch.from_numpy(v)], 1).bfloat16().cuda()
        qa.kv_write(both[:, H:2 * H], both[:, 2 * H:], cache, ints(slots))
    got = tensors(cache)
    for name, x, codes, scales in (("k", k, got[0], got[1]), ("v", v, got[2], got[3])):
        rc, rs = kv_oracle.store(x, table)
        pc, ps = np.zeros_like(codes), np.zeros_like(scales)
        pc[slots[keep] // page, :, slots[keep] % page] = rc[keep]
        ps[slots[keep] // page, :, slots[keep] % page] = rs[keep]
        assert np.array_equal(scales, ps), f"{name}: scales differ"
        assert np.array_equal(codes, pc), f"{name}: codes differ"
    for dtype in (torch.float32, torch.bfloat16):
        for name, x, back in zip("kv", (k, v), qa.kv_read(cache, ints(slots), dtype)):
            ref = kv_oracle.values(*kv_oracle.store(x, table), table)
            ref = np.where(keep[:, None, None], ref, 0.0).astype(np.float32)
            if dtype == torch.float32:
                assert np.array_equal(host(back), ref), f"{name}: fp32 values differ"
            else:
                assert np.array_equal(host_bf16_bits(back) & 0x7FFF, kv_oracle.bf16_bits(ref) & 0x7FFF), name
                assert np.array_equal(bf16_f64(host_bf16_bits(back)), bf16_f64(kv_oracle.bf16_bits(ref))), name


def test_many_bf16_tokens_are_exact():
    test_store_and_read_back_are_exact(0, 1031, 40, 128, 64, False)


@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
def test_a_run_with_a_non_finite_element_reads_back_as_nan(bad):
    x = np.random.default_rng(1).normal(0, 1, (3, 2, 128)).astype(np.float32)
    x[1, 0, 70] = bad
    cache = qa.kv_cache(1, 16, 2, 128)
    qa.kv_write(dev_f32(x), dev_f32(x), cache, ints([3, 4, 5]))
    ref = kv_oracle.values(*kv_oracle.store(x, 0), 0).astype(np.float32)
    assert np.isnan(ref[1, 0, 64:]).all() and np.isfinite(ref).sum() == ref.size - 64
    for back in qa.kv_read(cache, ints([3, 4, 5]), torch.float32):
        assert np.array_equal(host(back), ref, equal_nan=True)


def test_no_tokens():
    cache = qa.kv_cache(2, 16, 2, 64)
    none = torch.empty((0, 2, 64), device="cuda")
    qa.kv_write(none, none, cache, ints([]))
    k, v = qa.kv_read(cache, ints([]))
    assert k.shape == v.shape == (0, 2, 64)
    out, lse = qa.kv_attention(torch.empty((0, 4, 64), dtype=torch.bfloat16, device="cuda"), cache, ints([[0, 1]]),
                               ints([5]), want_lse=True)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)


# ------------------------------------------------------------------ attention

def filled_cache(rng, pages, page, H, D, table, gain=1.0):
    """Every row holds a token; codes and scale bits are drawn, not stored."""
    codes = [rng.integers(0, 256, (pages, H, page, D // 2), dtype=np.uint8) for _ in range(2)]
    scales = [kv_oracle.bf16_bits((gain * np.exp(rng.normal(0, 0.5, (pages, H, page, D // 64)))).astype(np.float32))
              for _ in range(2)]
    return codes, scales


def check(out, ref, spread, size, name):
    d = 2.0 ** -10 * size[..., None]
    tol = 2.0 ** -8 * np.abs(ref) + (np.expm1(2 * d) + 3 * 2.0 ** -11 + 2.0 ** -20) * spread
    bad = ~(np.abs(out - ref) <= tol)
    assert not bad.any(), f"{name}: {bad.sum()} of {bad.size} outputs off, worst {np.nanmax(np.abs(out - ref) - tol):.3e}"


def run_case(seed, lengths, queries, Hkv, G, D, page, table, causal=True, window=0, uniform=False, gain=1.0,
             max_len=None, poison=True, hide=None, strided=False, scale=None, spoil=None, spike=None):
    """One attention call against the oracle.  Rows no sequence holds are poisoned with NaN scales.
    hide: (sequence, page) whose table entry is not a page.  spoil: (sequence, positions) stored as NaN."""
    rng = np.random.default_rng(seed)
    lengths, queries = list(lengths), list(queries)
    need = [-(-t // page) for t in lengths]
    pages = sum(need) + 3
    codes, scales = filled_cache(rng, pages, page, Hkv, D, table, gain)
    order = rng.permutation(pages)
    width = max(need + [1]) + 1
    bt = np.full((len(lengths), width), -1, np.int32)
    bt[:, -1] = 2 ** 31 - 1
    held = np.zeros((pages, page), bool)
    at = 0
    for b, n in enumerate(need):
        bt[b, :n] = order[at:at + n]
        at += n
        for t in range(lengths[b]):
            held[bt[b, t // page], t % page] = True
    if poison:
        for s in scales:
            s.transpose(0, 2, 1, 3)[~held] = np.uint16(0x7FC0)
    if spoil is not None:
        for t in spoil[1]:
            for s in scales:
                s[bt[spoil[0], t // page], :, t % page] = np.uint16(0x7FC0)
    if spike is not None:                                     # (sequence 0's position, factor)
        for s in scales:
            r = s[bt[0, spike[0] // page], :, spike[0] % page]
            s[bt[0, spike[0] // page], :, spike[0] % page] = kv_oracle.bf16_bits(kv_oracle.bits_f64(r) * spike[1])
    if hide is not None:
        bt[hide[0], hide[1]] = pages + 5
    starts = np.concatenate([[0], np.cumsum(queries)])
    T, Hq = int(starts[-1]), Hkv * G
    qb = kv_oracle.bf16_bits(rng.normal(0, 1, (T, Hq, D)).astype(np.float32))
    q = dev_bf16(qb)
    if strided:
        q = torch.cat([q, torch.full((T, 3, D), float("nan"), dtype=q.dtype, device="cuda")], 1)[:, :Hq]
    cache = qa.KVCache(torch.from_numpy(codes[0]).cuda(), dev_bf16(scales[0]), torch.from_numpy(codes[1]).cuda(),
                       dev_bf16(scales[1]), table)
    out, lse = qa.kv_attention(q, cache, ints(bt), ints(lengths), None if uniform else ints(starts),
                               None if uniform else max(queries + [0]), max_len, scale, causal, window, want_lse=True)
    torch.cuda.synchronize()
    out, lse = bf16_f64(host_bf16_bits(out)), host(lse).astype(np.float64)
    err = norm = 0.0
    for b, (length, n) in enumerate(zip(lengths, queries)):
        if n == 0:
            continue
        t = np.arange(length)
        pg = bt[b, t // page]
        absent = (pg < 0) | (pg >= pages)
        pg = np.where(absent, 0, pg)
        k, v = (kv_oracle.values(codes[i][pg, :, t % page], scales[i][pg, :, t % page], table) for i in range(2))
        ref, rlse, spread, size = kv_oracle.attend(kv_oracle.bits_f64(qb[starts[b]:starts[b + 1]]), k, v,
                                                   D ** -0.5 if scale is None else scale, causal, window,
                                                   absent)
        got, glse = out[starts[b]:starts[b + 1]], lse[starts[b]:starts[b + 1]]
        empty = np.isinf(rlse) & (rlse < 0)
        assert np.array_equal(glse == -np.inf, empty), f"sequence {b}: empty rows"
        assert not got[empty].any(), f"sequence {b}: rows that see nothing are not zero"
        seen_nan = np.isnan(rlse)
        assert np.isnan(got[seen_nan]).all() and np.isnan(glse[seen_nan]).all()
        ok = ~empty & ~seen_nan
        check(got[ok], ref[ok], spread[ok], size[ok], f"sequence {b}")
        assert np.all(np.abs(glse[ok] - rlse[ok]) <= 2.0 ** -10 * size[ok] + 2.0 ** -20 * (1 + np.abs(rlse[ok]))), b
        err += np.sum((got[ok] - ref[ok]) ** 2)
        norm += np.sum(ref[ok] ** 2)
    assert err <= FRO_TOL ** 2 * norm
    return out


EDGE_LENGTHS = [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 129, 255, 257, 511, 513, 700]


@pytest.mark.parametrize("table", [0, 1, 2])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_single_tokens(D, table):
    run_case(100 + D + table, EDGE_LENGTHS, [1] * len(EDGE_LENGTHS), 2, 4, D, 16 if D == 128 else 48, table, uniform=True)


@pytest.mark.parametrize("G", [1, 3, 7, 8, 16, 17, 33, 71])
def test_query_heads_on_a_shared_head(G):
    run_case(200 + G, [0, 1, 77, 300], [1] * 4, 2, G, 128, 32, 0, uniform=True, strided=True)


@pytest.mark.parametrize("D,G,n", [(64, 8, 5), (128, 1, 2), (128, 4, 9), (128, 2, 31), (256, 3, 11), (256, 1, 16)])
@pytest.mark.parametrize("window", [0, 1, 40])
def test_a_few_queries_each(D, G, n, window):
    run_case(300 + D + G, [n, n + 1, 64, 333, 0, n - 1], [n] * 6, 2, G, D, 16, 0, window=window, uniform=True)


@pytest.mark.parametrize("D,Hkv,G", [(64, 2, 1), (64, 1, 6), (128, 1, 1), (128, 2, 4), (256, 1, 2), (256, 2, 1)])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 33), (False, 100), (True, 1)])
def test_prompts(D, Hkv, G, causal, window):
    run_case(400 + D + G, [200, 65, 1, 129, 310], [200, 64, 1, 0, 130], Hkv, G, D, 32, G % 3, causal=causal,
             window=window)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_more_queries_than_tokens(D):
    run_case(500 + D, [3, 0, 70], [10, 5, 150], 1, 2, D, 16, 0)
    run_case(510 + D, [3, 0, 70], [10, 5, 150], 1, 2, D, 16, 0, causal=False, window=4)


@pytest.mark.parametrize("n", [1, 3, 100])
def test_long_sequences(n):
    run_case(600 + n, [5000, 9001], [n, n], 1, 2, 128, 64, 0, uniform=True)
    run_case(610 + n, [9001, 12], [n, min(n, 12)], 1, 2, 64, 256, 1, window=3000)


@pytest.mark.parametrize("n", [1, 300])
def test_very_long_context_of_stored_tokens(n):
    """Over 262144 stored normal tokens a result is a few hundredths of the values it averages: an error of the levels
    that has a mean over their codes would stand out against it."""
    T, D, page = 262144, 64, 256
    g = torch.Generator("cuda").manual_seed(11)
    cache = qa.kv_cache(T // page, page, 1, D)
    slots = torch.randperm(T // page, generator=g, device="cuda")[:, None] * page + torch.arange(page, device="cuda")
    k, v = (torch.randn((T, 1, D), generator=g, device="cuda") for _ in range(2))
    qa.kv_write(k, v, cache, slots.flatten().int())
    k, v = (x.double()[:, 0] for x in qa.kv_read(cache, slots.flatten().int(), torch.float32))
    q = torch.randn((n, 1, D), generator=g, device="cuda").bfloat16()
    out, lse = qa.kv_attention(q, cache, (slots[:, 0] // page).int()[None], ints([T]), causal=False, want_lse=True)
    score = q[:, 0].double() @ k.T.contiguous() * D ** -0.5
    ref, rlse = torch.softmax(score, -1) @ v, torch.logsumexp(score, -1)
    assert float((out[:, 0].double() - ref).norm() / ref.norm()) <= FRO_TOL
    assert float((lse[:, 0].double() - rlse).abs().max()) <= 1e-4


@pytest.mark.parametrize("n", [1, 80])
def test_length_past_max_len_is_read_whole(n):
    run_case(700 + n, [900, 100], [n, n], 2, 1, 128, 16, 0, uniform=True, max_len=100)


@pytest.mark.parametrize("n", [1, 80])
def test_positions_without_a_page_are_seen_by_nobody(n):
    for page in (16, 64):
        run_case(800 + n, [400, 333], [n, n], 2, 2, 128, page, 0, uniform=True, hide=(0, 2))
    run_case(810 + n, [90, 10], [n, 1], 1, 2, 64, 128, 0, hide=(0, 0))


@pytest.mark.parametrize("D,n", [(64, 7), (128, 7), (256, 7), (64, 150), (128, 150), (256, 150)])
def test_non_finite_positions_reach_only_the_queries_that_see_them(D, n):
    # positions length - 3 and length - 2 are seen by the last three queries only
    out = run_case(900 + D + n, [300], [n], 2, 2, D, 32, 0, uniform=True, spoil=(0, [297, 298]))
    assert np.isfinite(out[:n - 3]).all() and np.isnan(out[n - 3:]).all()


@pytest.mark.parametrize("n", [1, 120])
@pytest.mark.parametrize("gain", [2.0 ** -90, 2.0 ** -20, 2.0 ** 12, 2.0 ** 60])
def test_magnitudes(n, gain):
    run_case(1000 + n, [150, 61], [n, min(n, 61)], 1, 2, 128, 16, 0, gain=gain, scale=128 ** -0.5 / gain)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n", [1, 90])
def test_one_large_position(D, n):
    """One position's scales far above the rest, wherever it lies in a tile."""
    for at in (0, 5, 19, 37, 50, 77, 101, 140):
        run_case(1050 + at, [150], [n], 1, 1, D, 16, 0, causal=False, spike=(at, 2.0 ** 18),
                 scale=D ** -0.5 * 2.0 ** -18)


# ------------------------------------------------------------------ batches that fill the device

# The kernel is chosen by its estimated time: on an MI355X's 256 CUs these batches are large
# enough for tiles of 32, and of 256, query rows.  (kv heads, lengths, queries)
LARGE = {32: (32, [333, 77, 5, 40], [40, 33, 1, 40]), 256: (48, [333, 77, 3, 60], [130, 77, 3, 40])}
LARGE_KERNELS = [(64, 32), (128, 32), (64, 256), (128, 256), (256, 256)]


@pytest.mark.parametrize("D,rows", LARGE_KERNELS)
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 33), (False, 100), (True, 1)])
def test_large_batches(D, rows, causal, window):
    heads, lengths, queries = LARGE[rows]
    run_case(1300 + D + rows, lengths, queries, heads, 1, D, 16 if causal else 48, D // 64 % 3, causal=causal,
             window=window, strided=window == 33)


@pytest.mark.parametrize("D,Hkv,G,n", [(64, 20, 3, 100), (64, 10, 7, 90), (128, 16, 3, 90), (128, 12, 8, 40),
                                       (256, 8, 5, 110), (256, 3, 32, 30)])
def test_large_batches_on_shared_heads(D, Hkv, G, n):
    run_case(1320 + D + G, [310, 64, 1, 0, n], [n, 64, 1, 2, n - 5], Hkv, G, D, 32, 0)


@pytest.mark.parametrize("D,rows", LARGE_KERNELS)
def test_large_batches_without_some_pages(D, rows):
    heads, lengths, queries = LARGE[rows]
    run_case(1340 + D + rows, lengths, queries, heads, 1, D, 16, 0, hide=(0, 2))
    run_case(1341 + D + rows, lengths, queries, heads, 1, D, 128, 0, hide=(1, 0), window=60)


@pytest.mark.parametrize("D,rows", LARGE_KERNELS)
def test_large_batches_with_non_finite_positions(D, rows):
    heads, _, queries = LARGE[rows]
    n = queries[0]
    out = run_case(1360 + D + rows, [300, 300, 150], [n, n, 40], heads, 1, D, 32, 0, spoil=(0, [297, 298]))
    assert np.isfinite(out[:n - 3]).all() and np.isnan(out[n - 3:n]).all() and np.isfinite(out[n:]).all()


@pytest.mark.parametrize("D,rows", LARGE_KERNELS)
@pytest.mark.parametrize("gain", [2.0 ** -90, 2.0 ** 60])
def test_large_batches_magnitudes(D, rows, gain):
    heads, lengths, queries = LARGE[rows]
    run_case(1380 + D + rows, lengths, queries, heads, 1, D, 16, 0, gain=gain, scale=D ** -0.5 / gain)


@pytest.mark.parametrize("D,rows", LARGE_KERNELS)
@pytest.mark.parametrize("at", [0, 19, 37, 77, 140])
def test_large_batches_one_large_position(D, rows, at):
    heads, _, queries = LARGE[rows]
    n = queries[0]
    run_case(1400 + at + rows, [150, 140, 60], [n, n, 40], heads, 1, D, 16, 0, causal=False, spike=(at, 2.0 ** 18),
             scale=D ** -0.5 * 2.0 ** -18)


@pytest.mark.parametrize("D,Hkv,n", [(64, 16, 513), (128, 16, 260), (256, 8, 260)])
@pytest.mark.parametrize("window", [0, 700])
def test_prompts_with_their_positions_split(D, Hkv, n, window):
    """The first sequence's rows have several splits to join, some of the second's one, the last's none."""
    run_case(1440 + D, [1500, 700, 0], [n, n - 30, 1], Hkv, 1, D, 64, 0, window=window)


@pytest.mark.parametrize("D,Hkv,G", [(64, 2, 4), (64, 24, 2), (128, 2, 1), (128, 1, 40), (128, 48, 1), (256, 2, 3)])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 50)])
def test_prompts_and_steps_in_one_batch(D, Hkv, G, causal, window):
    """Few tokens for the sequences and the longest one's queries: two passes, whose border is at 16 query rows."""
    step = max(1, 16 // G)
    queries = [130, 1, step, step + 1, 0, 2, 1] + [1] * 9 + [40]
    lengths = [max(n, x) for n, x in zip(queries, [333, 1, 77, 64, 5, 0, 100] + [17 * i for i in range(9)] + [200])]
    run_case(1480 + D + G, lengths, queries, Hkv, G, D, 16, 0, causal=causal, window=window, hide=(0, 3))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_prompts_and_steps_with_their_positions_split(D):
    run_case(1500 + D, [3000, 5000, 40, 1, 2600, 0, 0, 0, 300], [280, 1, 3, 1, 1, 0, 0, 0, 9], 4, 2, D, 64, 0)
    run_case(1510 + D, [100] * 70 + [400, 900] + [30] * 5, [1] * 70 + [300, 200] + [3] * 5, 1, 4, D, 16, 0)


@pytest.mark.parametrize("D,G,long", [(64, 1, 90), (128, 4, 300), (256, 2, 90)])
def test_a_few_prompts_among_many_steps(D, G, long):
    """Prompts far apart in a batch of more sequences than a wave looks at at once, the first and the last among them."""
    queries = [40] + [1] * 253 + [long, 0, 37] + [1] * 300 + [31]
    run_case(1520 + D, [n + 5 * (n > 1) + 3 for n in queries], queries, 1, G, D, 16, 0)


def test_wide_heads_with_many_splits():
    run_case(1460, [6000, 2500], [1, 1], 2, 3, 256, 64, 0, uniform=True)


def test_strides_and_other_streams():
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run_case(1100, [100, 40], [30, 1], 2, 2, 128, 16, 0, strided=True)


def _decode_step(seed, B, Hkv, G, D, page, width, n):
    rng = np.random.default_rng(seed)
    codes, scales = filled_cache(rng, B * width, page, Hkv, D, 0)
    cache = qa.KVCache(torch.from_numpy(codes[0]).cuda(), dev_bf16(scales[0]), torch.from_numpy(codes[1]).cuda(),
                       dev_bf16(scales[1]))
    bt = ints(rng.permutation(B * width).reshape(B, width))
    x = rng.normal(0, 1, (B * n, Hkv * (G + 2), D)).astype(np.float32)
    return cache, bt, torch.from_numpy(x).bfloat16().cuda()


@pytest.mark.parametrize("n,length", [(1, 40), (1, 700), (60, 700)])
def test_graph_replay_matches_eager(n, length):
    B, Hkv, G, D, page, width = 3, 2, 4, 128, 16, 50
    cache, bt, x = _decode_step(1200 + n, B, Hkv, G, D, page, width, n)
    lengths = torch.full((B,), length, dtype=torch.int32, device="cuda")
    slots = torch.empty(B * n, dtype=torch.int32, device="cuda")
    ws = qa.kv_attention_workspace(cache, Hkv * G, B * n, B, n, width * page)

    def place():
        pos = (lengths[:, None] - n + torch.arange(n, device="cuda")).long()
        slots.copy_((bt.gather(1, pos // page).long() * page + pos % page).int().flatten())

    def step():
        qa.kv_write(x[:, Hkv * G:Hkv * (G + 1)], x[:, Hkv * (G + 1):], cache, slots)
        return qa.kv_attention(x[:, :Hkv * G], cache, bt, lengths, workspace=ws)[0]
    place()
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for r in range(4):
        lengths += 7 * r - 5
        x.mul_(0.75).add_(0.01 * r)
        place()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), step().view(torch.int16)), r
        torch.cuda.synchronize()


def test_results_repeat_bit_for_bit():
    for n, length in ((1, 900), (70, 900)):
        cache, bt, x = _decode_step(1300 + n, 2, 2, 4, 128, 16, 64, n)
        lengths = ints([length, length - 331])
        outs = [qa.kv_attention(x[:, :8], cache, bt, lengths, want_lse=True) for _ in range(4)]
        for o, lse in outs[1:]:
            assert torch.equal(o.view(torch.int16), outs[0][0].view(torch.int16)) and torch.equal(lse, outs[0][1])


def test_offsets_past_32_bits():
    """A cache whose codes pass 4 GiB a tensor: tokens stored, read and attended at its far end."""
    H, D, page = 2, 128, 256
    pages = (5 << 30) // (H * page * D // 2)
    cache = qa.kv_cache(pages, page, H, D)
    rng = np.random.default_rng(5)
    T = 600
    far = np.array([pages - 1, pages - 2, 1], np.int32)
    t = np.arange(T)
    slots = far[t // page].astype(np.int64) * page + t % page
    assert int(slots[0]) * H * D // 2 > 2 ** 32
    k, v = (rng.normal(0, 1, (T, H, D)).astype(np.float32) for _ in range(2))
    qa.kv_write(dev_f32(k), dev_f32(v), cache, ints(slots))
    kd, vd = (kv_oracle.values(*kv_oracle.store(x, 0), 0) for x in (k, v))
    for x, ref in zip(qa.kv_read(cache, ints(slots), torch.float32), (kd, vd)):
        assert np.array_equal(host(x), ref.astype(np.float32))
    for n in (1, 100):
        qb = kv_oracle.bf16_bits(rng.normal(0, 1, (n, 4, D)).astype(np.float32))
        out, _ = qa.kv_attention(dev_bf16(qb), cache, ints(far[None]), ints([T]))
        ref, _, spread, size = kv_oracle.attend(kv_oracle.bits_f64(qb), kd, vd, D ** -0.5, True, 0)
        check(bf16_f64(host_bf16_bits(out)), ref, spread, size, "far pages")


def test_decoder_block_steps_match_one_prompt():
    """The example's block: tokens taken one at a time against the whole sequence taken as one prompt.

    Both see the same codes except where rounding in the projections differs by the path its row count takes: an
    output of the q|k|v projection that lies within its rounding of a code's edge may take the next code.  With bf16
    outputs (2^-9 relative rms) and 16 levels about 0.1 apart that is about one element in 30, each moved by about 0.1
    of its run's scale, so a value moves by 2 % rms where it happens, 0.4 % on the whole; the o projection keeps
    relative sizes.  Bound: 5 times that."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decode_attention.py")
    spec = importlib.util.spec_from_file_location("decode_attention", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    assert example.run(seqs=2, prompt=150, steps=3) <= 2e-2


def test_a_forked_sequence_goes_on_like_its_origin():
    import os
    import runpy
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decode_attention.py")
    assert runpy.run_path(path)["run_forked"](prompt=131, steps=3) == 0.0


@pytest.mark.parametrize("table", [0, 1, 2])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_storing_what_was_read_back_gives_the_same_values(D, table):
    """The same scales, and the same codes but for FP4's, of whose two zeros the storing rule takes one."""
    T, H = 97, 3
    rng = np.random.default_rng(1600 + D + table)
    x = (rng.normal(0, 1, (2, T, H, D)) * np.exp(rng.normal(0, 3, (2, T, H, 1)))).astype(np.float32)
    first, second = (qa.kv_cache(-(-T // 16), 16, H, D, table=table) for _ in range(2))
    slots = ints(rng.permutation(T))
    qa.kv_write(dev_f32(x[0]), dev_f32(x[1]), first, slots)
    k, v = qa.kv_read(first, slots, torch.float32)
    qa.kv_write(k, v, second, slots)
    for name, a, b in zip(("k_codes", "k_scales", "v_codes", "v_scales"), tensors(first), tensors(second)):
        if table != 2 or name.endswith("scales"):
            assert np.array_equal(a, b), name
    for a, b in zip((k, v), qa.kv_read(second, slots, torch.float32)):
        assert np.array_equal(host(a), host(b))


@pytest.mark.parametrize("seed", range(24))
def test_seeded_shapes(seed):
    rng = np.random.default_rng(9000 + seed)
    D, page = int(rng.choice([64, 128, 256])), int(rng.choice([16, 32, 48, 80, 128, 256]))
    Hkv, G = int(rng.integers(1, 4)), int(rng.choice([1, 2, 3, 4, 5, 8]))
    B = int(rng.integers(1, 5))
    lengths = [int(np.exp(rng.uniform(0, np.log(900)))) for _ in range(B)]
    top = int(rng.choice([1, 4, 20, 200]))
    queries = [int(rng.integers(0, min(t, top) + 1)) for t in lengths]
    run_case(9100 + seed, lengths, queries, Hkv, G, D, page, int(rng.integers(0, 3)), bool(rng.random() < 0.8),
             int(rng.choice([0, 0, 5, 70, 400])), strided=bool(rng.random() < 0.5))


# ------------------------------------------------------------------ refusals

def test_refusals():
    cache = qa.kv_cache(4, 16, 2, 128)
    x = torch.zeros((3, 2, 128), device="cuda")
    q = torch.zeros((3, 4, 128), dtype=torch.bfloat16, device="cuda")
    bt, ln = ints([[0, 1]]), ints([5])
    with pytest.raises(ValueError):
        qa.kv_cache(4, 24, 2, 128)
    with pytest.raises(ValueError):
        qa.kv_cache(4, 16, 2, 96)
    with pytest.raises(ValueError):
        qa.KVCache(cache.k_codes, cache.k_scales[:2], cache.v_codes, cache.v_scales)
    with pytest.raises(ValueError):
        qa.kv_write(x.half(), x.half(), cache, ints([0, 1, 2]))
    with pytest.raises(ValueError):
        qa.kv_write(x, x.bfloat16(), cache, ints([0, 1, 2]))
    with pytest.raises(ValueError):
        qa.kv_write(x, x[:2], cache, ints([0, 1, 2]))
    with pytest.raises(ValueError):
        qa.kv_write(x, x, cache, ints([0, 1]))
    with pytest.raises(ValueError):
        qa.kv_write(x, x, cache, ints([0, 1, 2]).long())
    with pytest.raises(ValueError):
        qa.kv_write(x.transpose(1, 2).contiguous().transpose(1, 2), x, cache, ints([0, 1, 2]))
    with pytest.raises(ValueError):
        qa.kv_read(cache, ints([0]), torch.float16)
    with pytest.raises(ValueError):
        qa.kv_attention(q.float(), cache, bt, ln)
    with pytest.raises(ValueError):
        qa.kv_attention(q[..., :64], cache, bt, ln)
    with pytest.raises(ValueError):
        qa.kv_attention(q, cache, bt, ints([5, 5]))
    with pytest.raises(ValueError):
        qa.kv_attention(q, cache, bt, ln, q_starts=ints([0, 3]))
    with pytest.raises(qa.QLoraError):                         # 3 query heads on 2
        qa.kv_attention(q[:, :3], cache, bt, ln)
    with pytest.raises(qa.QLoraError):                         # 3 tokens on 2 sequences
        qa.kv_attention(q, cache, ints([[0], [1]]), ints([5, 5]))
    with pytest.raises(qa.QLoraError):
        qa.kv_attention(q, cache, bt, ln, window=-1)
    torch.cuda.synchronize()

"""8 bits with one float32 scale per block of 128 on the device: codes and scales bit for bit those of the
definition (the same float32 quotients and product), the values back, rows packed by expert."""
import numpy as np
import pytest
import torch

from moe_expert_ffn_03_gb300 import binding as B, build
from oracle import fp8_block as fb
from rowcheck import f64

pytestmark = pytest.mark.gpu

U8, F32, BF16 = torch.uint8, torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()


def values(rows, cols, dtype, seed, pad=0):
    """Values over many binades with zeros, a block of zeros and tiny ones, in a tensor of row pitch cols + pad."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.full((rows, cols + pad), float("nan"), dtype=dtype, device="cuda")
    v = torch.randn(rows, cols, generator=g, device="cuda") * torch.exp(3 * torch.randn(rows, 1, generator=g, device="cuda"))
    v[torch.rand(rows, cols, generator=g, device="cuda") < 0.1] = 0.0
    if rows > 2:
        v[1] = 0.0
        v[2] *= 2.0 ** -120
    t[:, :cols] = v.to(dtype)
    return t[:, :cols]


def fresh(rows, cols, blocks, tiles):
    e = lambda *s, dt=F32: torch.full(s, 77, dtype=dt, device="cuda")  # noqa: E731
    cb = -(-cols // 128)
    return (e(rows, cols, dt=U8), e(cb, rows), e(blocks * 128, cols, dt=U8), e(blocks, cb if tiles else cols))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("split,cols,pad", [([1], 1, 0), ([1], 128, 0), ([5, 0, 3], 8, 0), ([129, 128, 127], 136, 8),
                                            ([0, 40, 300], 130, 3), ([1, 0, 2, 3], 264, 0), ([700], 1003, 0), ([64] * 20, 392, 0), ([0] * 199 + [2] * 57, 72, 0)])
def test_quantize(split, cols, pad, dtype):
    rows = sum(split)
    extra = 5                                                # rows of no expert
    v = values(rows + extra, cols, dtype, cols + rows, pad)
    ss = torch.tensor(split, dtype=torch.int32, device="cuda")
    blocks = B.fp8_blocks(rows + extra, len(split))
    host = v[:rows].float().cpu().numpy()
    ref_c, ref_s = fb.rows8(host)
    for tiles in (False, True):
        c, s, tc, ts = fresh(rows + extra, cols, blocks, tiles)
        B.moe_fp8_block_quantize(v, c, s, ss, tc, ts, "tiles" if tiles else "tokens")
        assert np.array_equal(c[:rows].cpu().numpy(), ref_c) and np.array_equal(s[:, :rows].cpu().numpy(), ref_s)
        assert bool((c[rows:] == 77).all()) and bool((s[:, rows:] == 77).all()), "rows of no expert were written"
        rc, rs = fb.tokens8(host, split, tiles)
        used = rs.shape[0]
        assert np.array_equal(tc[: used * 128].cpu().numpy(), rc) and np.array_equal(ts[:used].cpu().numpy(), rs)
        assert bool((tc[used * 128:] == 77).all()) and bool((ts[used:] == 77).all()), "blocks of no expert were written"
        # one format alone gives the same
        c2, s2, tc2, ts2 = fresh(rows + extra, cols, blocks, tiles)
        B.moe_fp8_block_quantize(v, c2, s2, ss)
        B.moe_fp8_block_quantize(v, None, None, ss, tc2, ts2, "tiles" if tiles else "tokens")
        assert torch.equal(c, c2) and torch.equal(s, s2) and torch.equal(tc, tc2) and torch.equal(ts, ts2)
        # values back
        for dt in (F32, BF16):
            out = torch.zeros(rows, cols + 8, dtype=dt, device="cuda")[:, :cols]
            B.moe_fp8_block_dequantize(c[:rows].contiguous(), s[:, :rows].contiguous(), "rows", out)
            ref = torch.tensor(fb.rows_back(ref_c, ref_s)).float().to(dt)
            assert torch.equal(out.cpu(), ref)
            out = torch.zeros(used * 128, cols, dtype=dt, device="cuda")
            if used:
                B.moe_fp8_block_dequantize(tc[: used * 128], ts[:used].contiguous(), "tiles" if tiles else "tokens", out)
                ref = torch.tensor((fb.tiles_back if tiles else fb.tokens_back)(rc, rs)).float().to(dt)
                assert torch.equal(out.cpu(), ref)
    # without experts all rows are written
    c, s, _, _ = fresh(rows + extra, cols, blocks, False)
    B.moe_fp8_block_quantize(v, c, s)
    rc, rs = fb.rows8(v.float().cpu().numpy())
    assert np.array_equal(c.cpu().numpy(), rc) and np.array_equal(s.cpu().numpy(), rs)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("E,N,K", [(1, 1, 1), (3, 128, 128), (2, 130, 257), (4, 300, 136)])
def test_weights(E, N, K, dtype):
    w = values(E * N, K, dtype, N + K).view(E, N, K)
    c = torch.full((E, N, K), 77, dtype=U8, device="cuda")
    s = torch.full((E, -(-N // 128), -(-K // 128)), 77.0, device="cuda")
    B.moe_fp8_block_quantize_weights(w, c, s)
    back = torch.zeros(E, N, K, dtype=F32, device="cuda")
    B.moe_fp8_block_dequantize(c, s, "tiles", back)
    for e in range(E):
        rc, rs = fb.tiles8(w[e].float().cpu().numpy())
        assert np.array_equal(c[e].cpu().numpy(), rc) and np.array_equal(s[e].cpu().numpy(), rs)
        assert np.array_equal(back[e].cpu().numpy(), fb.tiles_back(rc, rs).astype(np.float32))


def test_ties_and_the_largest_value():
    """Rows whose largest magnitude is 448 have factor 1: every E4M3 value, and every tie between two."""
    vals = fb.E4M3[:127]
    row = np.zeros(256, dtype=np.float32)
    row[:127], row[127], row[128:254], row[254], row[255] = vals, -448, (vals[:-1] + vals[1:]) / 2, 448, -1
    v = torch.tensor(np.stack([row, -row]), device="cuda")
    c, s = torch.zeros(2, 256, dtype=U8, device="cuda"), torch.zeros(2, 2, device="cuda")
    B.moe_fp8_block_quantize(v, c, s)
    assert bool((s == 1).all()) and np.array_equal(c.cpu().numpy(), fb.encode(v.cpu().numpy()))
    assert list(c[0, :127].cpu()) == list(range(127))


def test_not_finite():
    """A NaN or an Inf takes its own block along, in each format, and nothing else."""
    v = values(200, 300, BF16, 3).contiguous()
    v[7, 5], v[8, 290], v[150, 131] = float("nan"), float("inf"), float("-inf")
    ss = torch.tensor([140, 60], dtype=torch.int32, device="cuda")
    host = v.float().cpu().numpy()
    for tiles in (False, True):
        c, s, tc, ts = fresh(200, 300, B.fp8_blocks(200, 2), tiles)
        B.moe_fp8_block_quantize(v, c, s, ss, tc, ts, "tiles" if tiles else "tokens")
        rc, rs = fb.rows8(host)
        assert np.array_equal(c.cpu().numpy(), rc) and np.array_equal(s.cpu().numpy(), rs)
        rc, rs = fb.tokens8(host, [140, 60], tiles)
        assert np.array_equal(tc.cpu().numpy(), rc) and np.array_equal(ts.cpu().numpy(), rs)
        assert not bool(tc[140:256].any()) and not bool(tc[256 + 60:].any())           # rows behind the experts' last


@pytest.mark.parametrize("split", [[5, -1], [5, 60], [2 ** 31 - 1, 2 ** 31 - 1]])
def test_inconsistent_sizes_write_nothing(split):
    v = values(40, 64, BF16, 1)
    c, s, tc, ts = fresh(40, 64, B.fp8_blocks(40, 2), False)
    B.moe_fp8_block_quantize(v, c, s, torch.tensor(split, dtype=torch.int32, device="cuda"), tc, ts)
    for t in (c, s, tc, ts):
        assert bool((t == 77).all())


@pytest.mark.parametrize("T,k,E,cols", [(1, 1, 1, 16), (5, 2, 8, 128), (300, 8, 256, 144), (700, 3, 40, 1040)])
def test_pack(T, k, E, cols):
    g = torch.Generator(device="cuda").manual_seed(T)
    c = torch.randint(0, 255, (T, cols), generator=g, device="cuda").to(U8)
    s = torch.rand(-(-cols // 128), T, generator=g, device="cuda")
    idx = torch.rand(T, E, generator=g, device="cuda").topk(k, 1).indices.to(torch.int32)
    prob = torch.rand(T, k, generator=g, device="cuda")
    flat = idx.flatten().long()
    split = torch.bincount(flat, minlength=E).to(torch.int32)
    order = torch.argsort(flat, stable=True)                 # rows by expert, tokens in order
    pos = torch.empty_like(order)
    pos[order] = torch.arange(T * k, device="cuda")
    pad = torch.cumsum((split + 127) // 128 * 128, 0) - (split + 127) // 128 * 128
    first = torch.cumsum(split, 0) - split
    row_of = (pos + (pad - first)[flat]).to(torch.int32).view(T, k)
    ws = torch.zeros(256, dtype=U8, device="cuda")

    def run():
        out = [torch.full((T * k, cols), 77, dtype=U8, device="cuda"), torch.full((s.shape[0], T * k), 77.0, device="cuda"),
               torch.full((T * k,), 77.0, device="cuda"), torch.full((T, k), 77, dtype=torch.int32, device="cuda")]
        B.moe_fp8_block_pack(c, s, idx, prob, row_of, split, *out, ws)
        return out

    co, so, pr, po = run()
    assert B.moe_get_device_error(ws) == (0, 0) and torch.equal(po.flatten().long(), pos)
    tok = order // k
    assert torch.equal(co, c[tok]) and torch.equal(so, s[:, tok]) and torch.equal(pr, prob.flatten()[order])
    # a row that is none of its expert's is recorded and skipped
    lost = int(pos[0])
    row_of[0, 0] += 1000000
    co2, so2, pr2, po2 = run()
    assert B.moe_get_device_error(ws)[0] == 7 and int(po2[0, 0]) == -1
    keep = [i for i in range(T * k) if i != lost]
    assert torch.equal(co2[keep], co[keep]) and torch.equal(so2[:, keep], so[:, keep]) and torch.equal(pr2[keep], pr[keep])
    assert bool((co2[lost] == 77).all()) and float(pr2[lost]) == 77.0 and bool((so2[:, lost] == 77).all())


def test_values_are_exact_products():
    """A value is one float32 product: code times scale."""
    c = torch.arange(256, device="cuda").to(U8).repeat(4, 1).contiguous()
    s = torch.rand(2, 4, device="cuda") + 0.1
    out = torch.zeros(4, 256, device="cuda")
    B.moe_fp8_block_dequantize(c, s, "rows", out)
    ref = fb.E4M3[c.cpu().numpy()].astype(np.float32) * np.repeat(s.t().cpu().numpy(), 128, axis=1)
    assert np.array_equal(f64(out), ref.astype(np.float64), equal_nan=True)


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("rows,cols", [(1, 9), (3, 11), (700, 129), (301, 134), (37, 135), (301, 137), (64, 1003), (5, 3829), (9000, 255)])
def test_values_of_rows_of_any_length(rows, cols, dt):
    """Rows and tiles that start anywhere, blocks of one value, of seven, of eight, several rows in a vector's eight values."""
    g = torch.Generator(device="cuda").manual_seed(rows + cols)
    c = torch.randint(0, 127, (rows, cols), generator=g, device="cuda").to(U8) | (torch.randint(0, 2, (rows, cols), generator=g, device="cuda") << 7).to(U8)
    cb, host = -(-cols // 128), c.cpu().numpy()
    s = torch.rand(cb, rows, generator=g, device="cuda") + 0.5
    out = torch.full((rows, cols), 77.0, dtype=dt, device="cuda")
    B.moe_fp8_block_dequantize(c, s, "rows", out)
    values = fb.E4M3[host].astype(np.float32)
    wide = np.repeat(s.cpu().numpy().T, 128, 1)[:, :cols]
    assert torch.equal(out.cpu(), torch.tensor(values * wide).to(dt))
    mats = next(n for n in (3, 2, 1) if rows % n == 0)       # weights: every matrix on blocks of its own
    m = rows // mats
    s = torch.rand(mats, -(-m // 128), cb, generator=g, device="cuda") + 0.5
    out = torch.full((mats, m, cols), 77.0, dtype=dt, device="cuda")
    B.moe_fp8_block_dequantize(c.view(mats, m, cols), s, "tiles", out)
    wide = np.repeat(np.repeat(s.cpu().numpy(), 128, 2)[:, :, :cols], 128, 1)[:, :m]
    assert torch.equal(out.cpu(), torch.tensor(values.reshape(mats, m, cols) * wide).to(dt))

"""paged_kv_write_rope against its formula in 64 bits.

The kernel computes in fp32 and rounds once. With y the normed row, the fp32 error of a rotated value is at most
d (|c y_a| + |s y_b|), d = (D / 2 + 12) 2^-24: a sum of D squares is off by D roundings of 2^-24 at most and its root by
half of that, rsqrtf by 2^-22 (4), and the weight's, root's and angle's products, their sum and its negation add few.
The output's rounding is half a step: eps / 2 of its value, or half the smallest step. An E4M3 code's quotient adds one
fp32 rounding."""
import pytest
import torch

from paged_kv_cache_91_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(autouse=True)
def clean_error_word(cuda_lib):
    binding.device_errors(clear=True)
    yield


def angles(most, R):
    a = torch.arange(most, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)
    return torch.cat([a.cos(), a.sin()], 1).float()


def make(seed, T, H, Hkv, D, B, dtype="bf16", fp8=False, R=None, norm="qk", fused=False, most=500, spare=3):
    g = torch.Generator().manual_seed(seed)
    dt = TYPES[dtype]
    R = D if R is None else R
    NB = -(-T // B) + spare
    qkv = torch.randn((T, H + 2 * Hkv, D), generator=g).to(dt)
    c = dict(T=T, H=H, Hkv=Hkv, D=D, B=B, R=R, dtype=dt, fp8=fp8, NB=NB, eps=1e-5)
    qkv = qkv.to(DEV)
    c["q"], c["k"], c["v"] = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
    if not fused:
        c["q"], c["k"], c["v"] = (c[n].contiguous() for n in "qkv")
    slots = torch.randperm(NB * B, generator=g)[:T]
    slots[torch.rand(T, generator=g) < 0.2] = -1
    c["slots"] = slots
    c["pos"] = torch.randint(0, most, (T,), generator=g, dtype=torch.int32) if R else None
    c["cs"] = angles(most, R) if R else None
    c["qw"] = 1 + 0.3 * torch.randn(D, generator=g) if "q" in norm else None
    c["kw"] = 1 + 0.3 * torch.randn(D, generator=g) if "k" in norm else None
    c["scales"] = (0.02, 0.015) if fp8 else ()
    shape = (NB, Hkv, B, D)
    if fp8:
        c["kc"], c["vc"] = (torch.randint(0, 256, shape, generator=g, dtype=torch.uint8) for _ in range(2))
    else:
        c["kc"], c["vc"] = (torch.randn(shape, generator=g).to(dt) for _ in range(2))
    return c


def on(x):
    return None if x is None else x.to(DEV)


def call(c, interleaved=False, out=None, **kw):
    out = torch.full((c["T"], c["H"], c["D"]), float("nan"), dtype=c["dtype"], device=DEV) if out is None else out
    kc, vc = c["kc"].to(DEV), c["vc"].to(DEV)
    fn = binding.paged_kv_write_rope_fp8 if c["fp8"] else binding.paged_kv_write_rope
    fn(out, c["q"], c["k"], c["v"], kc, vc, c["slots"].to(DEV), on(c["pos"]), on(c["cs"]), *c["scales"],
       q_weight=on(c["qw"]), k_weight=on(c["kw"]), eps=c["eps"], interleaved=interleaved, **kw)
    torch.cuda.synchronize()
    return out, kc.cpu(), vc.cpu()


def formula(c, x, weight, interleaved):
    """(value, the largest fp32 error) of rows x [T][heads][D]."""
    D, R = c["D"], c["R"]
    y = x.double().cpu()
    if weight is not None:
        y = y / (y.square().mean(-1, keepdim=True) + c["eps"]).sqrt() * weight.double()
    big = y.abs()
    if R:
        cs = c["cs"][c["pos"].clamp(0, c["cs"].shape[0] - 1).long()].double()[:, None]
        co, si = cs[..., :R // 2], cs[..., R // 2:]
        lo, hi = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
        a, b = y[..., lo].clone(), y[..., hi].clone()
        y, big = y.clone(), big.clone()
        y[..., lo], y[..., hi] = a * co - b * si, b * co + a * si
        big[..., lo], big[..., hi] = ((a * co).abs() + (b * si).abs(), (b * co).abs() + (a * si).abs())
    return y, (D / 2 + 12) * 2.0 ** -24 * big


def near(got, ref, err, eps, step):
    got, tol = got.double().cpu(), eps / 2 * (ref.abs() + err) + err + step / 2
    assert bool(torch.isfinite(got).all())
    assert not got.numel() or float(((got - ref).abs() / tol).max()) <= 1.0


def near16(c, got, x, weight, interleaved=False):
    fi = torch.finfo(c["dtype"])
    near(got, *formula(c, x, weight, interleaved), fi.eps, fi.smallest_normal * fi.eps)


def check(c, interleaved=False, **kw):
    before = c["kc"].clone(), c["vc"].clone()
    out, kc, vc = call(c, interleaved, **kw)
    fi = torch.finfo(c["dtype"])
    near16(c, out, c["q"], c["qw"], interleaved)
    k, kerr = formula(c, c["k"], c["kw"], interleaved)
    v = c["v"].double().cpu()
    has = c["slots"] >= 0
    blk, off = c["slots"][has] // c["B"], c["slots"][has] % c["B"]
    if c["fp8"]:
        for pool, x, err, s in ((kc, k, kerr, c["scales"][0]), (vc, v, 0 * v, c["scales"][1])):
            s = torch.tensor(s, dtype=torch.float32).double()  # the call's scale is an fp32 number
            ref, err = (x / s).clamp(-448, 448)[has], err[has] / s + 2.0 ** -24 * (x / s).abs()[has]
            near(pool[blk, :, off].view(torch.float8_e4m3fn), ref, err, 2.0 ** -3, 2.0 ** -9)
    else:
        near(kc[blk, :, off], k[has], kerr[has], fi.eps, fi.smallest_normal * fi.eps)
        assert torch.equal(vc[blk, :, off], c["v"].cpu()[has])
    for pool, old in zip((kc, vc), before):  # and nothing else is written
        old[blk, :, off] = pool[blk, :, off]
        assert torch.equal(pool, old)
    assert binding.device_errors() == 0


SHAPES = [(1, 1, 64, 8), (8, 2, 128, 16), (40, 40, 128, 16), (5, 3, 64, 32), (64, 8, 128, 32), (17, 1, 128, 8)]


@pytest.mark.parametrize("T", [1, 2, 7, 130, 700])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype,fp8", [("f16", False), ("bf16", False), ("f16", True), ("bf16", True)])
@pytest.mark.parametrize("H,Hkv,D,B", SHAPES)
def test_rope(H, Hkv, D, B, dtype, fp8, interleaved, T):
    check(make(3, T, H, Hkv, D, B, dtype, fp8, fused=T % 2 == 0), interleaved)


@pytest.mark.parametrize("R", [0, 16, 32, 48, 64, 80, 96, 112, 128])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("fp8", [False, True])
def test_part_of_a_head_is_rotated(R, interleaved, fp8):
    for D in (64, 128):
        if R <= D:
            check(make(4, 33, 6, 2, D, 16, fp8=fp8, R=R, fused=True), interleaved)


@pytest.mark.parametrize("norm", ["", "q", "k", "qk"])
@pytest.mark.parametrize("fp8", [False, True])
def test_norms_are_optional(norm, fp8):
    check(make(5, 50, 8, 2, 128, 16, "f16", fp8, norm=norm))
    check(make(5, 50, 8, 2, 128, 16, "f16", fp8, norm=norm, R=0))


def test_without_norm_or_rotation_the_rows_are_copied():
    c = make(6, 40, 4, 4, 128, 16, norm="", R=0)
    out, kc, _ = call(c)
    assert torch.equal(out, c["q"])
    has = c["slots"] >= 0
    assert torch.equal(kc[c["slots"][has] // 16, :, c["slots"][has] % 16], c["k"].cpu()[has])


@pytest.mark.parametrize("T", [1, 90])
def test_queries_in_place(T):
    c = make(7, T, 8, 2, 128, 16)
    was = c["q"].clone()
    call(c, out=c["q"])
    near16(c, c["q"], was, c["qw"])


def test_one_token_in_place_of_a_projection():
    """A single token's slices are contiguous whatever the stride between tokens would be."""
    c = make(7, 1, 8, 2, 128, 16, fused=True)
    was = c["q"].clone()
    call(c, out=c["q"])
    near16(c, c["q"], was, c["qw"])


def test_extreme_rows():
    """Rows of zeros, of large values (whose squares fp32 holds) and of tiny ones; a NaN stays in its row."""
    c = make(8, 5, 2, 2, 128, 16, "f16")
    c["slots"] = torch.arange(5)
    for x in (c["q"], c["k"]):
        x[0], x[1], x[2] = 0.0, 30000.0, 6e-8
    check(c)
    c["q"][3, 1, 5] = float("nan")
    c["k"][4, 0, 7] = float("nan")
    out, kc, _ = call(c)
    nan = torch.isnan(out).any(-1).cpu()
    assert nan.nonzero().tolist() == [[3, 1]] and bool(torch.isnan(out[3, 1]).all())
    assert torch.isnan(kc[0, :, :5]).any(-1).nonzero().tolist() == [[0, 4]]


def test_saturating_codes():
    c = make(9, 20, 2, 2, 128, 16, fp8=True, norm="")
    c["k"] *= 40
    c["v"] *= 40
    check(c)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T", [3, 700])
def test_bad_positions_and_slots(T, fp8):
    """A position without angles: zeros, nothing stored, an error if the token has a slot. A slot past the pool:
    nothing stored, an error."""
    c = make(10, T, 8, 2, 128, 16, fp8=fp8)
    c["slots"] = torch.arange(T)
    fi = torch.finfo(c["dtype"])
    ref, err = formula(c, c["q"], c["qw"], False)
    c["pos"][0], c["pos"][2] = -1, 500
    for slot, error in ((0, 2), (-1, 0)):
        c["slots"][0] = c["slots"][2] = slot
        out, kc, vc = call(c)
        assert binding.device_errors(clear=True) == error
        assert not out[0].any() and not out[2].any()
        near(out[1], ref[1], err[1], fi.eps, fi.smallest_normal * fi.eps)
        for row in (0, 2):
            assert torch.equal(kc[0, :, row], c["kc"][0, :, row]) and torch.equal(vc[0, :, row], c["vc"][0, :, row])
    c["pos"][0] = c["pos"][2] = 3
    c["slots"][0], c["slots"][2] = c["NB"] * 16, 1 << 40
    ref, err = formula(c, c["q"], c["qw"], False)
    out, kc, vc = call(c)
    assert binding.device_errors(clear=True) == 4
    near(out, ref, err, fi.eps, fi.smallest_normal * fi.eps)
    for row in (0, 2):
        assert torch.equal(kc[0, :, row], c["kc"][0, :, row]) and torch.equal(vc[0, :, row], c["vc"][0, :, row])


def test_no_tokens():
    call(make(11, 0, 8, 2, 128, 16))
    assert binding.device_errors() == 0


def test_far_slots():
    """A pool of more than 2^31 elements, written at its end; and offsets of tokens that pass 2^31 bytes."""
    H, Hkv, D, B = 1, 8, 128, 32
    NB = (1 << 31) // (Hkv * B * D) + 3
    c = make(12, 6, H, Hkv, D, B)
    c["slots"] = NB * B - 1 - torch.arange(6)
    pools = [torch.zeros((NB, Hkv, B, D), dtype=c["dtype"], device=DEV) for _ in range(2)]
    out = torch.empty((6, H, D), dtype=c["dtype"], device=DEV)
    wide = torch.zeros((6, (1 << 28) + 8), dtype=c["dtype"], device=DEV)  # 2^29 bytes between tokens
    q = wide[:, :H * D].unflatten(1, (H, D))
    q.copy_(c["q"])
    binding.paged_kv_write_rope(out, q, c["k"], c["v"], *pools, c["slots"].to(DEV), on(c["pos"]), on(c["cs"]),
                                q_weight=on(c["qw"]), k_weight=on(c["kw"]), eps=c["eps"])
    torch.cuda.synchronize()
    near16(c, out, c["q"], c["qw"])
    blk, off = c["slots"].to(DEV) // B, c["slots"].to(DEV) % B
    near16(c, pools[0][blk, :, off], c["k"], c["kw"])
    assert torch.equal(pools[1][blk, :, off], c["v"])


def test_captured_and_on_another_stream():
    c = make(13, 64, 8, 2, 128, 16)
    want = call(c)
    out, kc, vc = torch.empty_like(want[0]), c["kc"].to(DEV), c["vc"].to(DEV)
    args = (out, c["q"], c["k"], c["v"], kc, vc, c["slots"].to(DEV), on(c["pos"]), on(c["cs"]))
    kw = dict(q_weight=on(c["qw"]), k_weight=on(c["kw"]), eps=c["eps"])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    binding.paged_kv_write_rope(*args, **kw, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(kc.cpu(), want[1]) and torch.equal(vc.cpu(), want[2])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        binding.paged_kv_write_rope(*args, **kw)
    for t in (out, kc, vc):
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0])
    has = c["slots"] >= 0
    blk, off = c["slots"][has] // 16, c["slots"][has] % 16
    assert torch.equal(kc.cpu()[blk, :, off], want[1][blk, :, off])

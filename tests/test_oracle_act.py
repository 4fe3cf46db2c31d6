"""Pins of the activation oracle (CPU): the 8-bit format against an exhaustive
search over its codes, the norms' gradients against differences, and the weight
gradient against a loop."""
import numpy as np
import pytest

from oracle import act

TYPES = {"fp16": np.float16, "bf16": None}


def _as(x, dtype):
    """float64 values rounded to the type (bf16 by bits, nearest even)."""
    x = np.asarray(x, np.float64)
    if dtype == "fp16":
        with np.errstate(over="ignore"):
            return x.astype(np.float16).astype(np.float64)
    b = x.astype(np.float32).view(np.uint32).astype(np.uint64)
    b = ((b + 0x7FFF + ((b >> 16) & 1)) >> 16 << 16).astype(np.uint32)
    return b.view(np.float32).astype(np.float64)


def test_e4m3_values():
    assert act.e4m3_value(0x00) == 0 and act.e4m3_value(0x01) == 2.0 ** -9
    assert act.e4m3_value(0x08) == 2.0 ** -6 and act.e4m3_value(0x38) == 1.0
    assert act.e4m3_value(0x7E) == 448 and np.isnan(act.e4m3_value(0x7F))
    assert act.e4m3_value(0xB8) == -1.0
    import torch
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.array([act.e4m3_value(c) for c in range(256)]), want,
                          equal_nan=True)


def test_e4m3_encoding_is_the_nearest_code_with_ties_to_even():
    grid = act._E4M3
    mids = (grid[:-1] + grid[1:]) / 2
    y = np.concatenate([grid, mids, np.nextafter(mids, 0), np.nextafter(mids, 1e9),
                        [455.0, 463.0]])
    y = np.concatenate([y, -y])
    got = act._encode_e4m3(y)
    want = np.array([act._nearest_e4m3(v) for v in y], dtype=np.uint8)
    assert np.array_equal(got, want)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_store_rule(fmt, dtype):
    rng = np.random.default_rng(1)
    mag = 2.0 ** rng.integers(-30 if dtype == "fp16" else -140,
                              16 if dtype == "fp16" else 128, size=(200, 3, 1))
    with np.errstate(over="ignore"):
        x = _as((rng.standard_normal((200, 3, 32)) * mag).reshape(200, 96)[:, :77], dtype)
    x[~np.isfinite(x)] = 0.0
    codes, scales = act.store(x, fmt, dtype)
    h = act.held(codes, scales, fmt)
    assert np.array_equal(_as(h, dtype), h)            # representable in the type
    for t in range(0, 200, 5):
        for b in range(3):
            blk = x[t, 32 * b:32 * b + 32]
            hb = h[t, 32 * b:32 * b + 32]
            amax, s = np.abs(blk).max(), 2.0 ** (int(scales[t, b]) - 127)
            if fmt == "int8":
                assert scales[t, b] >= 1
                if scales[t, b] > 1:
                    assert 64 * s <= amax < 128 * s
                near = np.abs(blk) <= 127 * s
                assert np.all(np.abs(blk - hb)[near] <= s / 2)
                assert np.all(np.abs(blk - hb) < s)
            else:
                top = 1.875 * 2.0 ** act.E_MAX[dtype]
                held_max = min(amax, top)
                assert held_max <= 448 * s
                if scales[t, b] > 10:
                    assert held_max > 224 * s
                inside = np.abs(blk) <= top
                err = np.abs(blk - hb)[inside]
                assert np.all(err <= np.maximum(np.abs(blk[inside]) * 2.0 ** -4, s * 2.0 ** -10))


def test_store_special_blocks():
    x = np.zeros((4, 40))
    x[0, 3] = np.inf
    x[1, 35] = np.nan
    x[2, 0] = 65504.0
    for fmt in ("int8", "e4m3"):
        codes, scales = act.store(x, fmt, "fp16")
        h = act.held(codes, scales, fmt)
        assert scales[0, 0] == 255 and np.isnan(h[0, :32]).all() and (h[0, 32:] == 0).all()
        assert np.isnan(h[1, 32:]).all() and (h[1, :32] == 0).all()
        assert h[2, 0] == (127 * 512.0 if fmt == "int8" else 61440.0)
        assert (h[3] == 0).all()
    assert np.isnan(act.held(np.ones((1, 3), np.uint8), np.array([[255]], np.uint8), "int8")).all()
    assert (act.held(np.ones((1, 3), np.uint8), np.zeros((1, 1), np.uint8), "int8")
            == 2.0 ** -127).all()


def test_weight_grad_is_the_sum_over_tokens():
    rng = np.random.default_rng(2)
    dy, x = rng.standard_normal((5, 3)), rng.standard_normal((5, 4))
    want = np.zeros((3, 4))
    for t in range(5):
        for n in range(3):
            for k in range(4):
                want[n, k] += dy[t, n] * x[t, k]
    assert np.allclose(act.weight_grad(dy, x), want, rtol=1e-14, atol=1e-14)


@pytest.mark.parametrize("post", ["none", "rms", "layer"])
@pytest.mark.parametrize("pre", ["none", "rms", "layer"])
@pytest.mark.parametrize("gated", [False, True])
def test_gradients_against_differences(post, pre, gated):
    """Central differences of sum(out . a + z . c): second order in the step, so
    1e-6 leaves about 1e-12 of truncation and 1e-9 of rounding."""
    rng = np.random.default_rng(3)
    t, h, eps, scale = 3, 11, 1e-3, 0.7
    v = {"h": rng.standard_normal((t, h)), "b": rng.standard_normal((t, h))}
    if gated:
        v["g"] = rng.standard_normal((t, h))
    for name, kind in (("post", post), ("pre", pre)):
        if kind != "none":
            v["w_" + name], v["b_" + name] = rng.standard_normal(h), rng.standard_normal(h)
    a, c = rng.standard_normal((t, h)), rng.standard_normal((t, h))

    def norms(u):
        return tuple((k, eps, u.get("w_" + n), u.get("b_" + n))
                     for n, k in (("post", post), ("pre", pre)))

    def loss(u):
        o, z, _ = act.block_norm(u["h"], u["b"], *norms(u), gate=u.get("g"), scale=scale)
        return (o * a).sum() + ((z * c).sum() if pre != "none" else 0.0)

    out, z, st = act.block_norm(v["h"], v["b"], *norms(v), gate=v.get("g"), scale=scale)
    g = act.block_norm_grad(a, c if pre != "none" else None, out, v["b"], st, *norms(v),
                            gate=v.get("g"), scale=scale)
    names = {"h": "dres", "b": "dblock", "g": "dgate", "w_post": "dw_post", "b_post": "db_post",
             "w_pre": "dw_pre", "b_pre": "db_pre"}
    for k, x in v.items():
        num = np.zeros_like(x)
        for i in np.ndindex(x.shape):
            step = 1e-6
            up, dn = dict(v), dict(v)
            up[k], dn[k] = x.copy(), x.copy()
            up[k][i] += step
            dn[k][i] -= step
            num[i] = (loss(up) - loss(dn)) / (2 * step)
        assert np.allclose(g[names[k]], num, rtol=1e-6, atol=1e-7), k

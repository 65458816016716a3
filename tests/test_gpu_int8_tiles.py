"""Every tile shape of the int8 product, named by the kernel that ran (the library's own launch
records), at row counts, column counts and K that end inside a tile, a 16-byte-chunk step or a K piece.

The reference is an fp64 product of the codes on the device: its sums of integers below 2^53 are
exact, so the tolerance is that of tests/test_gpu_int8.py: three fp32 roundings, and half a bf16 step.
"""
import numpy as np
import pytest
import torch

from mixture_experts_layer_07_amd import binding as B
from mixture_experts_layer_07_amd.configs import INT8_CONFIGS
from test_gpu_int8 import check_rows, layer_of, offsets_of, weights_of, workspace
import oracle as orc

pytestmark = pytest.mark.gpu

# rows of each expert, N, K, kernel suffix ("" = 256-row tiles)
TILES = {
    "few-1": ([1], 4099, 1040, "_few"),
    "few-2-experts": ([0, 40, 1, 0, 33], 330, 2064, "_few"),
    "few-4": ([61], 130, 4000, "_few"),
    "few-8-small-grid": ([127], 1025, 1936, "_few"),
    "few-8-large-grid": ([97], 4130, 528, "_few"),
    "few-32-weight-rows": ([15], 6161, 1040, "_few"),
    "few-32-weight-rows-groups": ([1, 0, 35, 2, 0, 17, 16, 1], 1330, 528, "_few"),
    "few-8-32-weight-rows": ([115], 8290, 272, "_few"),
    "few-1-long": ([9], 1030, 4112, "_few"),
    "few-1-long-32-weight-rows": ([5], 6501, 2064, "_few"),
    "few-1-two-per-cu": ([3], 5121, 2320, "_few"),
    "few-2-long-groups": ([2, 0, 17, 9, 1, 30] * 2, 3101, 2064, "_few"),
    "few-4-large-grid": ([50], 4130, 400, "_few"),
    "few-4-large-grid-32-weight-rows": ([61], 8301, 528, "_few"),
    "few-8-small-grid-32-weight-rows": ([99], 7001, 528, "_few"),
    "m64": ([140], 770, 400, "_m64"),
    "m64-K-pieces": ([300], 300, 7152, "_m64"),
    "m64-K-pieces-many-tiles": ([300], 900, 14416, "_m64"),
    "m64-K-pieces-groups": ([70, 0, 3, 65], 700, 14416, "_m64"),
    "m64-one-step": ([333], 1000, 112, "_m64"),
    "m64-groups": ([70, 0, 3, 129, 64, 65], 515, 2032, "_m64"),
    "m128": ([1000], 4097, 1296, "_m128"),
    "m128-K-pieces": ([1100], 1900, 14416, "_m128"),
    "m128-one-step": ([8000], 301, 48, "_m128"),
    "m128-groups": ([500, 0, 129, 1, 900, 128], 1500, 1424, "_m128"),
    "m256": ([5000], 3333, 784, ""),
    "m256-two-steps": ([4090], 4091, 240, ""),
    "m256-groups": ([1030, 0, 257, 900, 1, 31, 33, 65, 129, 1500] * 2, 3001, 1296, ""),
    "m256-heights": ([1100, 129, 160, 161, 191, 0, 192, 193, 256 + 129, 2 * 256 + 192, 256, 255, 128] * 2, 3333, 2064, ""),
    "m256-heights-two-steps": ([129, 150, 192, 193, 170, 256] * 6, 4001, 240, ""),
    "m256-K-pieces": ([4900], 4096, 16624, ""),
    "m32": ([1, 0, 40, 31, 7, 33, 20, 96] * 8, 2050, 1296, "_m32"),
    "m32-two-steps": ([3, 18, 32, 65] * 40, 600, 208, "_m32"),
    "m32-K-pieces": ([20] * 64, 2100, 16400, "_m32"),
}


def exact_product(x, xs, w, ws, counts):
    out = torch.full((x.shape[0], w.shape[1]), float("nan"), dtype=torch.float64, device="cuda")
    lo = 0
    for e, c in enumerate(counts):
        if c:
            z = torch.mm(x[lo:lo + c].double(), w[e].double().t().contiguous())
            out[lo:lo + c] = z * xs[lo:lo + c].double()[:, None] * ws[e].double()
        lo += c
    return out


@pytest.mark.parametrize("f32", [False, True], ids=["bf16", "f32"])
@pytest.mark.parametrize("name", list(TILES))
def test_tile_shape(name, f32):
    counts, N, K, suffix = TILES[name]
    rows, E = sum(counts), len(counts)
    print(f"tile shape {name} rows={rows} E={E} N={N} K={K} f32={f32}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(len(name) + K)
    rnd = lambda *s: torch.randint(-128, 128, s, generator=g, device="cuda", dtype=torch.int8)  # noqa: E731
    x, w = rnd(rows + 1, K), rnd(E, N, K)
    xs = torch.rand(rows + 1, generator=g, device="cuda") + 0.01
    ws = (torch.rand((E, N), generator=g, device="cuda") - 0.4) * 2.0 ** -10
    y = torch.full((rows + 1, N), -7.0, dtype=torch.float32 if f32 else torch.bfloat16, device="cuda")
    wsp = workspace()
    B.profile_reset()
    B.profile_enable(True)
    try:
        B.moe_gemm_int8(x, xs, w, ws, y, wsp, offsets=offsets_of(counts))
        B.moe_gemm_int8(x, xs, w, ws, y, wsp, offsets=offsets_of(counts))   # the workspace as the first call left it
        torch.cuda.synchronize()
    finally:
        B.profile_enable(False)
    ran = [k for k in B.profile_read() if k.startswith("gemm_i8")]
    B.profile_reset()
    assert ran == ["gemm_i8" + ("_f32out" if f32 else "") + suffix]
    assert (y[rows] == -7).all(), "a row in no group was written"
    ref = exact_product(x[:rows], xs, w, ws, counts)
    tol = (3 * 2.0 ** -24 + (0.0 if f32 else 2.0 ** -8)) * (1 + 2.0 ** -16)
    assert bool(((y[:rows].double() - ref).abs() <= tol * ref.abs()).all())


BASE = INT8_CONFIGS[9]
# the SwiGLU epilogue and the gathered rows on each tile shape: (layer, suffix)
SWIGLU = {
    "few": (BASE.scaled(T=12, H=640, I=384, E=12, K=5, n_group=1, topk_group=1, I_shared=0), "_few"),
    "few-long": (BASE.scaled(T=3, H=2176, I=128, E=12, K=5, n_group=1, topk_group=1, I_shared=0), "_few"),
    "few-long-groups": (BASE.scaled(T=12, H=2176, I=2304, E=12, K=5, n_group=1, topk_group=1, I_shared=0), "_few"),
    "m64": (BASE.scaled(T=60, H=896, I=384, E=8, K=4, n_group=1, topk_group=1, I_shared=0), "_m64"),
    "m128": (BASE.scaled(T=1300, H=1152, I=640, E=4, K=2, n_group=1, topk_group=1, I_shared=0), "_m128"),
    "m32": (BASE.scaled(T=100, H=2176, I=1152, E=48, K=8, n_group=1, topk_group=1, I_shared=0), "_m32"),
    "m256": (BASE.scaled(T=3900, H=1920, I=1920, E=5, K=2, n_group=1, topk_group=1, I_shared=0), ""),
    "m256-heights": (BASE.scaled(T=2640, H=1920, I=1920, E=64, K=4, n_group=1, topk_group=1, I_shared=0), ""),
}


@pytest.mark.parametrize("name", list(SWIGLU))
def test_swiglu_on_tile_shape(name):
    cfg, suffix = SWIGLU[name]
    print("int8 experts on tiles", name, flush=True)
    layer, x, ex, _ = layer_of(cfg)
    layer.y_perm.fill_(float("nan"))
    layer.route(x)
    layer.permute(x)
    B.profile_reset()
    B.profile_enable(True)
    try:
        layer.expert_ffn(x)
        torch.cuda.synchronize()
    finally:
        B.profile_enable(False)
    ran = sorted(k for k in B.profile_read() if k.startswith("gemm_i8"))
    B.profile_reset()
    assert ran == ["gemm_i8_down" + suffix, "gemm_i8_gateup_swiglu" + suffix]
    ids = layer.topk_ids.cpu().numpy().astype(np.int64)
    _, offsets, sp, _ = orc.permute(ids, cfg.E)
    rng = np.random.default_rng(1)
    rows = np.unique(np.concatenate([offsets[:-1][np.diff(offsets) > 0], offsets[1:][np.diff(offsets) > 0] - 1,
                                     rng.integers(0, cfg.P, 300)]))
    codes, scales = orc.quantize_rows_int8(x.float().cpu().numpy())
    xv = orc.dequantize_rows_int8(codes, scales)[sp[rows] // cfg.K]
    owner = np.searchsorted(offsets, rows, side="right") - 1
    assert torch.isfinite(layer.y_perm.float()).all()
    check_rows(layer.y_perm[torch.from_numpy(rows).cuda()].double().cpu().numpy(), xv, owner, weights_of(ex))

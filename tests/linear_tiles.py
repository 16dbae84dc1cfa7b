"""Sizes that reach every tile of the linear layer's matrix kernels, whole and in parts, and the plan each of
them gets (host only).  Used by the CPU test that holds the list to the plan and by the GPU test that runs it."""
import ctypes

from int6_weight_export_amd import pgq

TYPE = {"f32": pgq.PGQ_F32, "bf16": pgq.PGQ_BF16}
ACT = {"none": pgq.PGQ_ACT_NONE, "silu": pgq.PGQ_ACT_SILU}
AT = {n: (i + 1) << 44 for i, n in enumerate(("x", "codes", "scales", "y", "z", "residual", "dy", "dx", "dw", "dbias"))}


def forward_plan(M, N, K, y, residual):
    """(tile rows, tile columns, from codes, in parts, Y's type) of a forward call that keeps Z, or None off the tiles."""
    p = pgq.pgq_linear_fwd(M=M, N=N, K=K, x=AT["x"], ldx=K, codes=AT["codes"], ldc=K, scales=AT["scales"], y=AT["y"], ldy=N,
                           y_dtype=TYPE[y], z=AT["z"], ldz=N)
    if residual:
        p.residual, p.ldr, p.residual_dtype = AT["residual"], N, TYPE[residual]
    o = pgq.pgq_linear_plan()
    assert pgq.pgq_linear_forward_plan(ctypes.byref(p), ctypes.byref(o)) == pgq.PGQ_OK
    return (o.tile_rows, o.tile_cols, o.from_codes, o.parts > 1, y) if o.path == pgq.PGQ_LINEAR_TILES else None


def backward_plan(M, N, K, want, t, act):
    """(outputs, dX's tile, in parts, dW's tile, in parts, outputs' type) of a backward call from a bf16 dY."""
    p = pgq.pgq_linear_bwd(M=M, N=N, K=K, dy=AT["dy"], lddy=N, dy_dtype=pgq.PGQ_BF16, z=AT["z"], ldz=N, x=AT["x"], ldx=K,
                           codes=AT["codes"], ldc=K, scales=AT["scales"], lddx=K, dx_dtype=TYPE[t], lddw=K, dw_dtype=TYPE[t],
                           act=ACT[act])
    for k in want.split():
        setattr(p, k, AT[k])
    o = pgq.pgq_linear_plan()
    assert pgq.pgq_linear_backward_plan(ctypes.byref(p), ctypes.byref(o)) == pgq.PGQ_OK
    assert o.joint == (want == "dx dw dbias")
    return ((want, o.tile_rows, o.tile_cols, o.parts > 1, o.dw_rows, o.dw_cols, o.dw_parts > 1, t)
            if o.path == pgq.PGQ_LINEAR_TILES else None)


# ((M, N, K, Y's type, residual's type), plan)
FORWARD = [
    ((10948, 135, 20, "bf16", "bf16"), (128, 128, 0, False, "bf16")),
    ((11430, 159, 18, "f32", "f32"), (128, 128, 0, False, "f32")),
    ((3058, 65, 4633, "bf16", "bf16"), (128, 128, 0, True, "bf16")),
    ((2076, 70, 6202, "f32", "f32"), (128, 128, 0, True, "f32")),
    ((10914, 3376, 16, "bf16", "f32"), (128, 128, 1, False, "bf16")),
    ((11386, 272, 144, "f32", ""), (128, 128, 1, False, "f32")),
    ((67, 2912, 6192, "bf16", ""), (128, 128, 1, True, "bf16")),
    ((73, 6544, 2320, "f32", "bf16"), (128, 128, 1, True, "f32")),
    ((8815, 16, 2784, "bf16", ""), (128, 64, 0, True, "bf16")),
    ((4618, 16, 6080, "f32", "bf16"), (128, 64, 0, True, "f32")),
    ((11217, 641, 18, "bf16", ""), (256, 192, 0, False, "bf16")),
    ((9370, 794, 20, "f32", "bf16"), (256, 192, 0, False, "f32")),
    ((2344, 5072, 18, "bf16", "bf16"), (256, 256, 0, False, "bf16")),
    ((8697, 1474, 17, "f32", ""), (256, 256, 0, False, "f32")),
    ((33, 16, 16, "bf16", "f32"), (64, 128, 1, False, "bf16")),
    ((33, 16, 16, "f32", "f32"), (64, 128, 1, False, "f32")),
    ((74, 16, 784, "bf16", ""), (64, 128, 1, True, "bf16")),
    ((70, 16, 816, "f32", ""), (64, 128, 1, True, "f32")),
    ((75, 17, 22, "bf16", "f32"), (64, 64, 0, False, "bf16")),
    ((72, 17, 21, "f32", ""), (64, 64, 0, False, "f32")),
    ((36, 17, 1089, "bf16", "bf16"), (64, 64, 0, True, "bf16")),
    ((34, 18, 1097, "f32", ""), (64, 64, 0, True, "f32")),
    ((11461, 135, 6932, "f32", "bf16"), (256, 192, 0, True, "f32")),
    ((11833, 129, 8181, "bf16", ""), (256, 192, 0, True, "bf16")),
    ((16208, 416, 8048, "bf16", "f32"), (256, 256, 0, True, "bf16")),
    ((16298, 400, 8048, "f32", "bf16"), (256, 256, 0, True, "f32")),
    # the sizes of the models here, and generic wide layers
    ((16384, 528, 1584, "f32", "f32"), (256, 192, 0, False, "f32")),
    ((16384, 1584, 528, "bf16", ""), (256, 256, 0, False, "bf16")),
    ((8192, 8192, 4096, "bf16", ""), (256, 256, 0, False, "bf16")),
    ((2048, 4096, 1024, "bf16", "f32"), (128, 128, 1, False, "bf16")),
]

# ((M, N, K, outputs, their type, activation), plan)
BACKWARD = [
    ((17, 534, 5507, "dw", "bf16", "none"), ("dw", 0, 0, False, 128, 128, False, "bf16")),
    ((18, 5803, 521, "dw", "f32", "silu"), ("dw", 0, 0, False, 128, 128, False, "f32")),
    ((4018, 793, 84, "dw", "bf16", "silu"), ("dw", 0, 0, False, 128, 128, True, "bf16")),
    ((1309, 1742, 68, "dw", "f32", "silu"), ("dw", 0, 0, False, 128, 128, True, "f32")),
    ((18, 1425, 5690, "dw", "bf16", "none"), ("dw", 0, 0, False, 256, 192, False, "bf16")),
    ((17, 2637, 3212, "dw", "f32", "silu"), ("dw", 0, 0, False, 256, 192, False, "f32")),
    ((4542, 1728, 144, "dw", "bf16", "silu"), ("dw", 0, 0, False, 256, 192, True, "bf16")),
    ((719, 6336, 137, "dw", "f32", "silu"), ("dw", 0, 0, False, 256, 192, True, "f32")),
    ((17, 3888, 3152, "dw", "bf16", "silu"), ("dw", 0, 0, False, 256, 256, False, "bf16")),
    ((17, 1600, 8096, "dw", "f32", "silu"), ("dw", 0, 0, False, 256, 256, False, "f32")),
    ((1913, 6192, 416, "dw", "bf16", "silu"), ("dw", 0, 0, False, 256, 256, True, "bf16")),
    ((1165, 5888, 416, "dw", "f32", "silu"), ("dw", 0, 0, False, 256, 256, True, "f32")),
    ((17, 16, 16, "dw", "bf16", "silu"), ("dw", 0, 0, False, 64, 64, False, "bf16")),
    ((17, 16, 16, "dw", "f32", "none"), ("dw", 0, 0, False, 64, 64, False, "f32")),
    ((201, 16, 16, "dw", "bf16", "silu"), ("dw", 0, 0, False, 64, 64, True, "bf16")),
    ((133, 16, 16, "dw", "f32", "silu"), ("dw", 0, 0, False, 64, 64, True, "f32")),
    ((204, 16, 6976, "dx dw dbias", "bf16", "none"), ("dx dw dbias", 128, 128, False, 128, 128, False, "bf16")),
    ((277, 16, 5616, "dx dw dbias", "f32", "none"), ("dx dw dbias", 128, 128, False, 128, 128, False, "f32")),
    ((669, 16, 2320, "dx dw dbias", "bf16", "silu"), ("dx dw dbias", 128, 128, False, 128, 128, True, "bf16")),
    ((330, 16, 4688, "dx dw dbias", "f32", "silu"), ("dx dw dbias", 128, 128, False, 128, 128, True, "f32")),
    ((20, 1008, 3648, "dx dw dbias", "bf16", "silu"), ("dx dw dbias", 128, 128, True, 128, 128, False, "bf16")),
    ((20, 800, 4000, "dx dw dbias", "f32", "silu"), ("dx dw dbias", 128, 128, True, 128, 128, False, "f32")),
    ((2429, 3028, 65, "dx dw dbias", "bf16", "silu"), ("dx dw dbias", 128, 128, True, 128, 128, True, "bf16")),
    ((2067, 2259, 66, "dx dw dbias", "f32", "silu"), ("dx dw dbias", 128, 128, True, 128, 128, True, "f32")),
    ((439, 544, 7584, "dx dw dbias", "bf16", "silu"), ("dx dw dbias", 256, 192, False, 256, 192, False, "bf16")),
    ((452, 608, 7184, "dx dw dbias", "f32", "none"), ("dx dw dbias", 256, 192, False, 256, 192, False, "f32")),
    ((9037, 176, 160, "dx dw dbias", "bf16", "none"), ("dx dw dbias", 256, 192, False, 256, 192, True, "bf16")),
    ((10225, 176, 272, "dx dw dbias", "f32", "silu"), ("dx dw dbias", 256, 192, False, 256, 192, True, "f32")),
    ((144, 1760, 1312, "dx dw dbias", "bf16", "silu"), ("dx dw dbias", 256, 192, True, 256, 192, False, "bf16")),
    ((69, 1488, 3440, "dx dw dbias", "f32", "silu"), ("dx dw dbias", 256, 192, True, 256, 192, False, "f32")),
    ((1408, 3047, 133, "dx dw dbias", "bf16", "silu"), ("dx dw dbias", 256, 192, True, 256, 192, True, "bf16")),
    ((1664, 1856, 160, "dx dw dbias", "f32", "silu"), ("dx dw dbias", 256, 192, True, 256, 192, True, "f32")),
    ((672, 288, 7216, "dx dw dbias", "bf16", "none"), ("dx dw dbias", 256, 256, False, 256, 192, False, "bf16")),
    ((649, 264, 7950, "dx dw dbias", "f32", "none"), ("dx dw dbias", 256, 256, False, 256, 192, False, "f32")),
    ((5745, 80, 1088, "dx dw dbias", "bf16", "silu"), ("dx dw dbias", 256, 256, False, 256, 192, True, "bf16")),
    ((11973, 22, 521, "dx dw dbias", "f32", "none"), ("dx dw dbias", 256, 256, False, 256, 192, True, "f32")),
    ((535, 822, 8035, "dx dw dbias", "bf16", "silu"), ("dx dw dbias", 256, 256, False, 256, 256, False, "bf16")),
    ((516, 915, 7631, "dx dw dbias", "f32", "silu"), ("dx dw dbias", 256, 256, False, 256, 256, False, "f32")),
    ((5934, 134, 1156, "dx dw dbias", "bf16", "silu"), ("dx dw dbias", 256, 256, False, 256, 256, True, "bf16")),
    ((1697, 136, 4578, "dx dw dbias", "f32", "silu"), ("dx dw dbias", 256, 256, False, 256, 256, True, "f32")),
    ((151, 619, 7030, "dx dw dbias", "bf16", "silu"), ("dx dw dbias", 256, 256, True, 256, 192, False, "bf16")),
    ((129, 672, 6928, "dx dw dbias", "f32", "silu"), ("dx dw dbias", 256, 256, True, 256, 192, False, "f32")),
    ((1571, 1129, 779, "dx dw dbias", "bf16", "silu"), ("dx dw dbias", 256, 256, True, 256, 192, True, "bf16")),
    ((705, 2656, 464, "dx dw dbias", "f32", "silu"), ("dx dw dbias", 256, 256, True, 256, 192, True, "f32")),
    ((129, 848, 6496, "dx dw dbias", "bf16", "silu"), ("dx dw dbias", 256, 256, True, 256, 256, False, "bf16")),
    ((19, 7136, 2512, "dx dw dbias", "f32", "none"), ("dx dw dbias", 256, 256, True, 256, 256, False, "f32")),
    ((2949, 2704, 208, "dx dw dbias", "bf16", "silu"), ("dx dw dbias", 256, 256, True, 256, 256, True, "bf16")),
    ((1495, 2252, 245, "dx dw dbias", "f32", "silu"), ("dx dw dbias", 256, 256, True, 256, 256, True, "f32")),
    ((17, 16, 16, "dx dw dbias", "bf16", "none"), ("dx dw dbias", 64, 64, False, 64, 64, False, "bf16")),
    ((17, 16, 16, "dx dw dbias", "f32", "silu"), ("dx dw dbias", 64, 64, False, 64, 64, False, "f32")),
    ((260, 16, 16, "dx dw dbias", "bf16", "silu"), ("dx dw dbias", 64, 64, False, 64, 64, True, "bf16")),
    ((201, 16, 16, "dx dw dbias", "f32", "silu"), ("dx dw dbias", 64, 64, False, 64, 64, True, "f32")),
    ((20, 400, 16, "dx dw dbias", "bf16", "silu"), ("dx dw dbias", 64, 64, True, 64, 64, False, "bf16")),
    ((17, 288, 16, "dx dw dbias", "f32", "silu"), ("dx dw dbias", 64, 64, True, 64, 64, False, "f32")),
    ((651, 481, 17, "dx dw dbias", "bf16", "silu"), ("dx dw dbias", 64, 64, True, 64, 64, True, "bf16")),
    ((412, 336, 16, "dx dw dbias", "f32", "silu"), ("dx dw dbias", 64, 64, True, 64, 64, True, "f32")),
    ((11425, 16, 144, "dx", "bf16", "silu"), ("dx", 128, 128, False, 0, 0, False, "bf16")),
    ((8637, 16, 208, "dx", "f32", "silu"), ("dx", 128, 128, False, 0, 0, False, "f32")),
    ((69, 1218, 4448, "dx", "bf16", "silu"), ("dx", 128, 128, True, 0, 0, False, "bf16")),
    ((65, 2672, 1760, "dx", "f32", "silu"), ("dx", 128, 128, True, 0, 0, False, "f32")),
    ((2117, 5440, 16, "dx", "bf16", "silu"), ("dx", 128, 64, True, 0, 0, False, "bf16")),
    ((4199, 2176, 16, "dx", "f32", "silu"), ("dx", 128, 64, True, 0, 0, False, "f32")),
    ((8336, 16, 928, "dx", "bf16", "none"), ("dx", 256, 192, False, 0, 0, False, "bf16")),
    ((11006, 16, 683, "dx", "f32", "none"), ("dx", 256, 192, False, 0, 0, False, "f32")),
    ((6071, 5488, 144, "dx", "bf16", "silu"), ("dx", 256, 192, True, 0, 0, False, "bf16")),
    ((2963, 6398, 137, "dx", "f32", "silu"), ("dx", 256, 192, True, 0, 0, False, "f32")),
    ((10912, 16, 1008, "dx", "bf16", "none"), ("dx", 256, 256, False, 0, 0, False, "bf16")),
    ((6595, 16, 1760, "dx", "f32", "silu"), ("dx", 256, 256, False, 0, 0, False, "f32")),
    ((186, 7216, 7088, "dx", "f32", "silu"), ("dx", 256, 256, True, 0, 0, False, "f32")),
    ((17, 16, 16, "dx", "bf16", "none"), ("dx", 64, 64, False, 0, 0, False, "bf16")),
    ((18, 16, 16, "dx", "f32", "none"), ("dx", 64, 64, False, 0, 0, False, "f32")),
    ((19, 560, 16, "dx", "bf16", "silu"), ("dx", 64, 64, True, 0, 0, False, "bf16")),
    ((20, 384, 16, "dx", "f32", "silu"), ("dx", 64, 64, True, 0, 0, False, "f32")),
    ((15615, 4551, 469, "dx", "bf16", "silu"), ("dx", 256, 256, True, 0, 0, False, "bf16")),
    ((16384, 1584, 528, "dx dw dbias", "bf16", "silu"), ("dx dw dbias", 256, 192, False, 256, 192, True, "bf16")),
    ((8192, 4096, 4096, "dx dw dbias", "bf16", "none"), ("dx dw dbias", 256, 256, False, 256, 256, False, "bf16")),
]

"""Grouped products of many rows, as cases that must reach the kernel for pairs of SMs, and its arguments for them."""
from tests import batch_helpers as B

# name: group sizes, output columns, k.  Uneven groups with tails; columns whose halves of gate and up are no multiple of 16
# rows; one group of more row tiles than a band has; a short k; groups that end on and beside a tile's or a box's border
PAIR = {
    "uneven": ([0, 1, 37, 600, 255, 257, 513, 385], 1056, 2056),
    "by 16": ([300, 700, 0, 64], 1000, 2120),
    "bands": ([2400, 3], 1304, 2112),
    "short k": ([512, 700, 33, 800], 1536, 192),
    "borders": ([256, 512, 32, 64, 96, 1, 288, 31], 1040, 2072),
    "one column over": ([512, 511, 513], 3592, 2064),
}


def args(M, sizes, n, k, kn=False, swiglu=False, gather=False, scatter=False, out="bf16", dtype="bf16", pitch=8, m=None):
    """The arguments of a call on 16-byte aligned operands (an output pitch of n + pitch)."""
    code = {"bf16": M.T_BF16, "fp16": M.T_FP16, "fp32": M.T_FP32}
    m = sum(sizes) if m is None else m
    nw, p = n * (2 if swiglu else 1), 4096
    return M.GroupedArgs(x=p, w=p, offsets=p, rows=p if gather else None, out_rows=p if scatter else None, out=p, x_rows=m, ldx=k,
                         ldw=nw if kn else k, w_stride=nw * k, out_rows_n=m + 3, ldo=n + pitch, m=m, groups=len(sizes), n=nw, k=k,
                         dtype=code[dtype], out_dtype=code[out], layout=M.GROUP_KN if kn else M.GROUP_NK,
                         act=M.ACT_SWIGLU if swiglu else M.ACT_NONE, workspace=p if gather else None,
                         workspace_bytes=M.grouped_workspace(m, k, len(sizes)) if gather else 0)


def wgrad_args(M, sizes, n, k, out="bf16", dy_rows=False, x_rows=False):
    m, p = sum(sizes), 4096
    ws = (M.grouped_wgrad_workspace(m, n) if dy_rows else 0) + (M.grouped_wgrad_workspace(m, k) if x_rows else 0)
    return M.GroupedWgradArgs(dy=p, x=p, offsets=p, dy_rows=p if dy_rows else None, x_rows=p if x_rows else None, dw=p, dy_rows_n=m,
                              lddy=n, x_rows_n=m, ldx=k, lddw=k, dw_stride=n * k, m=m, groups=len(sizes), n=n, k=k, dtype=0,
                              out_dtype={"bf16": 0, "fp16": 1, "fp32": 2}[out], workspace=p if ws else None, workspace_bytes=ws)

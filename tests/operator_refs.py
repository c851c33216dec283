"""Plain float64 forms of the operators around the block, on the CPU, for the parity tests."""
import torch

DIM = 128


def column_blocks(cols):
    return [(j * DIM, min((j + 1) * DIM, cols)) for j in range(-(-cols // DIM))]


def rms_norm(x, weight, eps, residual=None):
    """(h, y) in float64 of bf16 / float32 inputs."""
    h = x.double() if residual is None else x.double() + residual.double()
    return h, h / torch.sqrt(h.square().mean(1, keepdim=True) + eps) * weight.double()


def e4m3_half_step(q):
    """Half the distance between neighbouring e4m3 values around each q (float64)."""
    e = torch.floor(torch.log2(q.abs().clamp_min(2.0 ** -6)))
    return torch.exp2(e - 4)


def e4m3_rne(q):
    """The e4m3 value nearest to each q, ties to even, at most 448 in magnitude."""
    step = 2 * e4m3_half_step(q)
    return (torch.round(q / step) * step).clamp(-448, 448)


def quantize(x, block_rows=1):
    """(codes as values, scales [column blocks, row blocks]) of a bf16 matrix by the definition:
    scale = max|x| / 448 in float32, code of the float32 quotient."""
    rows, cols = x.shape
    nr = -(-rows // block_rows)
    values = torch.empty((rows, cols), dtype=torch.float64)
    scales = torch.empty((-(-cols // DIM), nr), dtype=torch.float32)
    for j, (c0, c1) in enumerate(column_blocks(cols)):
        for i in range(nr):
            b = x[i * block_rows:(i + 1) * block_rows, c0:c1].float()
            a = b.abs().max()
            s = a / torch.tensor(448.0) if a > 0 else torch.tensor(1.0)
            scales[j, i] = s
            values[i * block_rows:(i + 1) * block_rows, c0:c1] = e4m3_rne((b / s).double())
    return values, scales


def gemm(a_values, a_scales, w_values, w_scales):
    """(out, sum of |terms|) in float64."""
    m, n = a_values.shape[0], w_values.shape[0]
    out = torch.zeros((m, n), dtype=torch.float64)
    mag = torch.zeros_like(out)
    for j, (c0, c1) in enumerate(column_blocks(a_values.shape[1])):
        s = a_scales[j].double()[:, None] * w_scales[j].double().repeat_interleave(DIM)[None, :n]
        a, w = a_values[:, c0:c1].double(), w_values[:, c0:c1].double()
        out += a @ w.t() * s
        mag += a.abs() @ w.abs().t() * s.abs()
    return out, mag

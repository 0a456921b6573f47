"""A layer's input rows kept in 8 bits between its forward pass and the step.

K-FAC needs a fully connected layer's input twice after the forward pass (Osawa et al., CVPR
2019, eq. 5 and 7): for the weight gradient g^T a that is preconditioned, and for the factor
A = E[a a^T]. A Checkpoint holds it as whole numbers of 8 bits with a power of two for each
row, half the memory of fp16; autograd and the step share it (what made the input may keep it
for a backward pass of its own, as a ReLU does). Its values are what both
are formed from (kfac_weight_grad_q8, kfac_factors_q8): s q is exact in 16 bits, so neither
rounds anything further. Every number is computed by libkfac; there is no CPU path.
"""
import torch
import torch.nn.functional as F
from torch.autograd.function import once_differentiable

from . import _lib as K


class Checkpoint:
    """Rows q [rows, cols] (int8) with a scale [rows] (float32) each, a power of two (with others a
    factor formed from it is NaN); a scale of 0 marks a row that takes no part (kfac.h)."""

    def __init__(self, q, scale):
        if q.dim() != 2 or q.dtype != torch.int8 or scale.dtype != torch.float32 or scale.shape != q.shape[:1]:
            raise TypeError("a checkpoint is int8 [rows, cols] with float32 [rows]")
        self.q, self.scale = q, scale

    @classmethod
    def of(cls, x, mask=None):
        """The checkpoint of x [rows, cols] in float16, bfloat16 or float32."""
        cp = cls.empty(x)
        K.kfac_quantize_rows(_rows(x), cp.q, cp.scale, mask=mask)
        return cp

    @classmethod
    def empty(cls, x):
        """Room for the checkpoint of x."""
        if x.dim() != 2:
            raise ValueError("a checkpoint takes rows: [rows, features]")
        return cls(torch.empty(x.shape, dtype=torch.int8, device=x.device),
                   torch.empty(x.shape[0], dtype=torch.float32, device=x.device))

    def values(self, dtype=torch.float32):
        """What the rows stand for."""
        x = torch.empty(self.q.shape, dtype=dtype, device=self.q.device)
        K.kfac_dequantize_rows(self.q, self.scale, x)
        return x

    # what the capture and the step ask of a tensor
    @property
    def shape(self):
        return self.q.shape

    @property
    def device(self):
        return self.q.device

    def __len__(self):
        return len(self.q)

    def index_select(self, dim, index):
        if dim != 0:
            raise ValueError("a checkpoint's rows are dimension 0")
        return Checkpoint(self.q.index_select(0, index), self.scale.index_select(0, index))


def _rows(x):
    """x as rows for the library: contiguous within, apart from each other."""
    if (x.shape[1] > 1 and x.stride(1) != 1) or (len(x) > 1 and x.stride(0) < x.shape[1]):
        return x.contiguous()
    return x


class _Linear(torch.autograd.Function):
    """x W^T + b whose backward pass takes x from a checkpoint."""

    @staticmethod
    def forward(ctx, x, weight, bias, cp, int8):
        if int8:
            y = linear_int8(x, weight, bias, cp)
        else:
            K.kfac_quantize_rows(_rows(x), cp.q, cp.scale)
            y = F.linear(x, weight, bias)
        ctx.save_for_backward(weight, cp.q, cp.scale)
        ctx.bias_dtype = None if bias is None else bias.dtype
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, g):
        weight, q, scale = ctx.saved_tensors
        need_x, need_w, need_b = ctx.needs_input_grad[:3]
        need_b = need_b and ctx.bias_dtype is not None
        gx = g @ weight if need_x else None
        dw = db = None
        if need_w or need_b:
            dw = torch.empty(weight.shape, dtype=torch.float32, device=g.device)
            db = torch.empty(len(weight), dtype=torch.float32, device=g.device) if need_b else None
            K.kfac_weight_grad_q8(_rows(g), q, scale, dw, dbias=db)
            dw = dw.to(weight.dtype) if need_w else None
            db = db.to(ctx.bias_dtype) if need_b else None
        return gx, dw, db, None, None


def linear_int8(x, weight, bias=None, cp=None):
    """x W^T + b in 8-bit integers (kfac_linear_q8), the weights quantised as they are at the call; the
    input's checkpoint goes into cp, if one is given."""
    cp = Checkpoint.empty(x) if cp is None else cp
    wq = torch.empty(weight.shape, dtype=torch.int8, device=weight.device)
    ws = torch.empty(len(weight), dtype=torch.float32, device=weight.device)
    K.kfac_quantize_rows(_rows(weight.detach()), wq, ws, pow2=False)
    y = torch.empty(len(x), len(weight), dtype=x.dtype, device=x.device)
    K.kfac_linear_q8(_rows(x), cp.q, cp.scale, wq, ws, y, bias=bias)
    return y


def linear(x, weight, bias=None, int8=False):
    """(x W^T + b, the checkpoint of x): a fully connected layer that keeps its input in 8 bits for
    its backward pass. int8: the product is formed in 8-bit integers too; the gradient at x
    is then g W with the weights as they are. Under autocast in its type."""
    if torch.is_autocast_enabled("cuda"):
        t = torch.get_autocast_dtype("cuda")
        x, weight, bias = x.to(t), weight.to(t), None if bias is None else bias.to(t)
    cp = Checkpoint.empty(x)
    with torch.autocast("cuda", enabled=False):
        return _Linear.apply(x, weight, bias, cp, int8), cp

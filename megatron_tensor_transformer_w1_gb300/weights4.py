"""Weights in four bits with a scale for each group of input features
(tp_quantize4, tp_*_shard_*4 of include/tpffn.h).

    codes = quantize4(W, group=128)                    # Codes4: codes and scales in the natural layout
    w13_4, w2_4 = ffn.pack4(W1, W2, W3, group=128)     # Packed4: what the passes read
    y = ffn.forward4(x, w13_4, w2_4)

PyTorch allocates the device buffers and supplies the stream; every step runs
in libtpffn.so.
"""
from __future__ import annotations

import threading

import torch

from . import tpffn as abi

GROUPS = (32, 64, 128)
BF16 = torch.bfloat16
current_device = torch._C._cuda_getDevice
current_stream = torch._C._cuda_getCurrentRawStream
_capturing = torch._C._cuda_isCurrentStreamCapturing


def check_tensor(name, t, dtype, shape, index):
    """Refuses what the library would read or write otherwise than meant; `index`
    is the CUDA device's."""
    if (not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.shape != shape or not t.is_contiguous()
            or t.get_device() != index):
        got = f"{t.dtype} {tuple(t.shape)} on {t.device}" if isinstance(t, torch.Tensor) else type(t).__name__
        raise ValueError(f"{name}: a contiguous {dtype} tensor of shape {tuple(shape)} on cuda:{index} is needed, not {got}")


def device_index(device):
    """The index of a CUDA device, the current one's where it names none."""
    device = torch.device(device)
    if device.type != "cuda":
        raise ValueError(f"a CUDA device is needed, not {device}")
    return current_device() if device.index is None else device.index


class Scratch:
    """Workspaces of one object's calls: one for every stream of a device that it has
    been used on; a call that is being captured into a graph takes its own, from the
    graph's memory.  Host threads on one stream take turns (`turn`), as the launches of
    a call follow one another in the stream's workspace."""

    def __init__(self):
        self.turn, self._kept = threading.Lock(), {}

    def take(self, nbytes, index, stream):
        if _capturing():
            return torch.empty(nbytes, dtype=torch.uint8, device=index)
        t = self._kept.get((index, stream))
        if t is None or t.numel() < nbytes:
            t = self._kept[index, stream] = torch.empty(nbytes, dtype=torch.uint8, device=index)
        return t


class Codes4:
    """A matrix [rows, cols] in 4-bit codes: codes uint8 [rows, (cols + 1) // 2] (the
    even column in a byte's low half) and scales bfloat16 [rows, segments *
    ceil(cols / segments / group)]; element (code - 8) * scale.  The groups start
    anew in each of `segments` equal parts of a row."""

    def __init__(self, codes, scales, cols, group=128, segments=1):
        cols, group, segments = int(cols), int(group), int(segments)
        if group not in GROUPS:
            raise ValueError(f"group is one of {GROUPS}, not {group}")
        if cols < 0 or segments < 1 or cols % segments:
            raise ValueError(f"{cols} columns are not {segments} equal segments")
        if not isinstance(codes, torch.Tensor) or codes.dim() != 2:
            raise ValueError("codes: a uint8 tensor [rows, (cols + 1) // 2] is needed")
        rows = codes.shape[0]
        index = codes.get_device()
        check_tensor("codes", codes, torch.uint8, (rows, (cols + 1) // 2), index)
        check_tensor("scales", scales, BF16, (rows, segments * -(-(cols // segments) // group)), index)
        self.codes, self.scales = codes, scales
        self.rows, self.cols, self.group, self.segments, self.device = rows, cols, group, segments, codes.device

    @classmethod
    def empty(cls, rows, cols, group, segments, index):
        if group not in GROUPS or segments < 1 or cols % segments:
            raise ValueError(f"group is one of {GROUPS}, and the columns ({cols}) are equal segments ({segments})")
        c = cls.__new__(cls)
        c.codes = torch.empty((rows, (cols + 1) // 2), dtype=torch.uint8, device=index)
        c.scales = torch.empty((rows, segments * -(-(cols // segments) // group)), dtype=BF16, device=index)
        c.rows, c.cols, c.group, c.segments, c.device = rows, cols, group, segments, c.codes.device
        return c


class Packed4:
    """Weights in the layout that the 4-bit passes read, of one sublayer and side
    (TP_PACK_COLUMNS or TP_PACK_ROWS)."""

    def __init__(self, data, group, which, key):
        self.data, self.group, self.which, self.key = data, group, which, key


def quantize4(W, group=128, segments=1):
    """W [rows, cols] bfloat16 as Codes4: scale bf16(max |w| / 7) for each group,
    code rint(w / scale) + 8."""
    if not isinstance(W, torch.Tensor) or W.dim() != 2 or not W.is_cuda:
        raise ValueError("W: a bfloat16 matrix on a CUDA device is needed")
    index = W.get_device()
    if current_device() != index:
        with torch.cuda.device(index):
            return quantize4(W, group, segments)
    check_tensor("W", W, BF16, W.shape, index)
    c = Codes4.empty(W.shape[0], W.shape[1], group, segments, index)
    rc = abi._lib.tp_quantize4(W.data_ptr(), c.rows, c.cols, segments, group, c.codes.data_ptr(), c.scales.data_ptr(),
                               current_stream(index))
    if rc:
        abi.check(rc, "tp_quantize4")
    return c


def dequantize4(c):
    """The matrix that a Codes4 stands for, bfloat16 [rows, cols]."""
    if not isinstance(c, Codes4) or not c.codes.is_cuda:
        raise ValueError("c: a Codes4 on a CUDA device is needed")
    index = c.codes.get_device()
    if current_device() != index:
        with torch.cuda.device(index):
            return dequantize4(c)
    W = torch.empty((c.rows, c.cols), dtype=BF16, device=index)
    rc = abi._lib.tp_dequantize4(c.codes.data_ptr(), c.scales.data_ptr(), c.rows, c.cols, c.segments, c.group, W.data_ptr(),
                                 current_stream(index))
    if rc:
        abi.check(rc, "tp_dequantize4")
    return W


def as_codes(name, W, rows, cols, group, segments, index):
    """W, a bfloat16 matrix or a Codes4, as the Codes4 that a sublayer wants."""
    if isinstance(W, Codes4):
        if (W.rows, W.cols, W.group, W.segments, W.codes.get_device()) != (rows, cols, group, segments, index):
            raise ValueError(f"{name}: codes of {rows} x {cols}, groups of {group}, {segments} segment(s) on cuda:{index} "
                             f"are needed, not of {W.rows} x {W.cols}, {W.group}, {W.segments} on {W.device}")
        return W
    check_tensor(name, W, BF16, (rows, cols), index)
    return quantize4(W, group, segments)


def group_of(group, *weights):
    """The group size of a pack: that of the codes given, else `group`, else 128."""
    sizes = {w.group for w in weights if isinstance(w, Codes4)} | ({int(group)} if group is not None else set())
    if len(sizes) > 1:
        raise ValueError(f"one group size is needed, not {sorted(sizes)}")
    size = sizes.pop() if sizes else 128
    if size not in GROUPS:
        raise ValueError(f"group is one of {GROUPS}, not {size}")
    return size


def check_packed(name, w, which, key, index, group=None):
    if not isinstance(w, Packed4) or w.which != which or w.key != key:
        raise ValueError(f"{name}: the 4-bit weight that this sublayer packed is needed")
    if w.data.get_device() != index or (group is not None and w.group != group):
        raise ValueError(f"{name}: a weight on cuda:{index} with the other's group size is needed")

"""Checks and pointers of tensor arguments, one pass per tensor (a decode step's call is paid mostly on the host).

Like the package's other entry points these refuse, before any launch, what the C ABI cannot see: a wrong element
type, shape, stride or device.  The device of the call is
the first tensor's, passed around as its index (tensor.get_device(): an integer, -1 for the CPU); stream() refuses
one that is no CUDA (HIP) device and comes last, so that a wrong type or shape is named first.
"""

import torch

U8 = (torch.uint8,)
F32 = (torch.float32,)
I64 = (torch.int64,)
HI = (torch.bfloat16, torch.float32)

_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def stream(device):
    """The current stream of the call's device, as an integer."""
    if device < 0:
        raise ValueError("the tensors must be on a CUDA (HIP) device")
    return _raw_stream(device) if _raw_stream is not None else torch.cuda.current_stream(device).cuda_stream


def _refuse(t, name, shape, dtypes, device):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must have dtype {' or '.join(str(d) for d in dtypes)}, not {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    raise ValueError(f"{name} is on {t.device}, the call's first tensor elsewhere")


def matrix(t, name, shape, dtypes, device):
    """(address, leading dimension) of a matrix of the given shape with unit column stride."""
    if not isinstance(t, torch.Tensor) or t.dtype not in dtypes or t.shape != shape or t.get_device() != device:
        _refuse(t, name, shape, dtypes, device)
    rows, cols = shape
    if rows == 0 or cols == 0:
        return t.data_ptr(), cols  # (an empty matrix has no meaningful strides; the call does nothing with it)
    ld, unit = t.stride()
    if unit != 1 and cols > 1:
        raise ValueError(f"{name}: expected a 2-D tensor with unit column stride")
    return t.data_ptr(), ld if rows > 1 else max(ld, cols)


def scale_words(t, name, shape, device):
    """(address, leading dimension in words) of scales [words, rows, 4]."""
    if not isinstance(t, torch.Tensor) or t.dtype not in U8 or t.shape != shape or t.get_device() != device:
        _refuse(t, name, shape, U8, device)
    words, rows, _ = shape
    if words == 0 or rows == 0:
        return t.data_ptr(), max(rows, 1)
    ld, row, unit = t.stride()
    if unit != 1 or (rows > 1 and row != 4) or (words > 1 and ld % 4):
        raise ValueError(f"{name}: scales must be [words, rows, 4] with rows of four bytes next to each other")
    return t.data_ptr(), ld // 4 if words > 1 else rows


NONE = (0, 0)  # of an output that is not wanted


def experts_of(offsets):
    """E of an offsets tensor of E + 1 entries."""
    if not isinstance(offsets, torch.Tensor):
        raise TypeError("offsets must be a torch tensor")
    if offsets.dim() != 1 or offsets.shape[0] < 2 or not offsets.is_contiguous():
        raise ValueError("offsets must be a contiguous 1-D tensor of E + 1 entries")
    return offsets.shape[0] - 1


def experts(offsets, device):
    """(address, E) of an offsets tensor of E + 1 entries."""
    E = experts_of(offsets)
    if offsets.dtype not in I64 or offsets.get_device() != device:
        _refuse(offsets, "offsets", offsets.shape, I64, device)
    return offsets.data_ptr(), E


def space(ws, device):
    """(address, bytes) of a workspace tensor or None."""
    if ws is None:
        return 0, 0
    if not isinstance(ws, torch.Tensor):
        raise TypeError("ws must be a torch tensor or None")
    if not ws.is_contiguous():
        raise ValueError("ws must be contiguous")
    if ws.get_device() != device:
        raise ValueError(f"ws is on {ws.device}, the call's tensors elsewhere")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def stacked(rows, E, what):
    """Rows per expert of `rows` stacked ones."""
    if rows % E:
        raise ValueError(f"{what}: {rows} stacked rows do not split over {E} experts")
    return rows // E

"""Checks and pointers of tensor arguments, one pass per tensor (a decode step's call is paid mostly on the host).

Like the package's other entry points these refuse, before any launch, what the C ABI cannot see: a wrong element
type, shape, stride or device.  The device of the call is
the first tensor's, passed around as its index (tensor.get_device(): an integer, -1 for the CPU); stream() refuses
one that is no CUDA (HIP) device and comes last, so that a wrong type or shape is named first.
"""

import functools

import torch

U8 = (torch.uint8,)
I8 = (torch.int8,)
I32 = (torch.int32,)
F32 = (torch.float32,)
BF16 = (torch.bfloat16,)
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


def flat(t, name, shape, dtypes, device):
    """Address of a contiguous tensor of the given shape."""
    if not isinstance(t, torch.Tensor) or t.dtype not in dtypes or t.shape != shape or t.get_device() != device:
        _refuse(t, name, shape, dtypes, device)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def vector(t, name, n, dtypes, device):
    """Address of a contiguous vector of n elements."""
    return flat(t, name, (n,), dtypes, device)


def batch(t, name, shape, dtypes, device):
    """(address, matrices, rows, columns, leading dimension, distance of matrices) of a matrix or a batch of them."""
    if not isinstance(t, torch.Tensor) or t.dtype not in dtypes or t.shape != shape or t.get_device() != device:
        _refuse(t, name, shape, dtypes, device)
    B, R, C = shape if len(shape) == 3 else (1, *shape)
    if t.numel() == 0:
        return t.data_ptr(), B, R, C, max(C, 1), max(R * C, 1)
    st = t.stride()
    if st[-1] != 1 and C > 1:
        raise ValueError(f"{name}: expected matrices with unit column stride")
    ld = st[-2] if R > 1 else C
    return t.data_ptr(), B, R, C, ld, st[0] if B > 1 else (R - 1) * ld + C


_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _any_tensor(kwargs):
    return next((v for v in kwargs.values() if isinstance(v, torch.Tensor)), None)


def on_its_device(fn):
    """fn(tensor, ...) with the tensor's device as the current one: plans, workspace sizes and launches go by that.  Where all
    arguments are named any tensor of them tells the device (tensors of two devices are refused)."""

    @functools.wraps(fn)
    def call(*args, **kwargs):
        first = args[0] if args else _any_tensor(kwargs)
        if not isinstance(first, torch.Tensor) or not first.is_cuda or first.get_device() == _current_device():
            return fn(*args, **kwargs)
        with torch.cuda.device(first.get_device()):
            return fn(*args, **kwargs)

    def prepared(launch, args, kwargs):
        device = (args[0] if args else _any_tensor(kwargs)).get_device()

        def there():
            if device == _current_device():
                launch()
            else:
                with torch.cuda.device(device):
                    launch()

        return there

    call.prepared = prepared  # (what prepare() makes of a launch of this call)
    return call


def stacked(rows, E, what):
    """Rows per expert of `rows` stacked ones."""
    if rows % E:
        raise ValueError(f"{what}: {rows} stacked rows do not split over {E} experts")
    return rows // E

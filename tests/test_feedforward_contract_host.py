"""What the feed-forward operators promise about their workspaces and check
about their arguments, without a GPU."""

import ctypes
import itertools

import pytest

torch = pytest.importorskip("torch")

import mixed_precision_optimizer_gb300 as mp
from mixed_precision_optimizer_gb300 import build_lib


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build_lib.build()


ROWS = [0, 1, 100, 256, 257, 2048, 8192, 16384, 16385, 100000]
ALIGNED = [16, 512, 1024, 2560, 4096, 5120, 9728, 14336, 19456, 77808, 77824, 128256]
ANY = [1, 7, 63, 777, 1023, 4097, 9727, 38911, 77823, 77825]


@pytest.mark.parametrize("any_layout", [False, True])
def test_linear_workspace_serves_smaller_sizes(any_layout):
    """A size is at least that of every call whose m, n and k are none larger:
    with any_layout for all widths, without it for those that need no copy."""
    widths = sorted(ALIGNED + ANY) if any_layout else ALIGNED
    size = {s: mp.linear_workspace_size(*s, any_layout=any_layout) for s in itertools.product(ROWS, widths, widths)}
    for axis in range(3):
        for s in size:
            values = (ROWS, widths, widths)[axis]
            i = values.index(s[axis])
            if i:                                    # one step down each axis: the rest follows
                smaller = s[:axis] + (values[i - 1],) + s[axis + 1:]
                assert size[smaller] <= size[s], (smaller, s)


def test_linear_workspace_of_every_width():
    """The same in steps of one column past each change of the slices, where
    the bias gradient's partial sums go up and down."""
    for m in (512, 8192, 16384):
        sizes = [mp.linear_workspace_size(m, n, 16, any_layout=True) for n in range(1, 20000, 7)]
        assert sizes == sorted(sizes)
    # aligned widths, and the two orders of a block's products
    assert mp.linear_workspace_size(8192, 128256, 4096) >= mp.linear_workspace_size(8192, 4096, 4096)
    assert mp.linear_workspace_size(8192, 9728, 2560) >= mp.linear_workspace_size(8192, 2560, 9728)
    assert mp.linear_workspace_size(128, 4096, 4096, any_layout=True) >= mp.linear_workspace_size(128, 4096, 1023)


# -------------------------------------------------------------- devices --

class OnDevice:
    """Stands in for a dense tensor on a device that this machine need not have."""

    def __init__(self, dtype, *shape, device=0, contiguous=True):
        self.dtype, self.shape, self._device, self._contiguous = dtype, torch.Size(shape), device, contiguous

    is_cuda = property(lambda self: self._device >= 0)
    device = property(lambda self: torch.device("cuda", self._device) if self._device >= 0 else torch.device("cpu"))

    def get_device(self):
        return self._device

    def stride(self):
        return tuple(self.shape[i + 1:].numel() for i in range(len(self.shape)))

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return torch.empty(0, dtype=self.dtype).element_size()

    def is_contiguous(self):
        return self._contiguous

    def data_ptr(self):
        return 1 << 20


BF, F32, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
T = OnDevice


def calls():
    """name -> (function, the tensors it takes by name, with a workspace that is large enough)"""
    ws = T(torch.uint8, 1 << 20)
    return {
        "rmsnorm": (mp.rmsnorm, dict(x=T(BF, 4, 64), gamma=T(BF, 64), residual=T(BF, 4, 64), h=T(BF, 4, 64), y=T(BF, 4, 64),
                                     q=T(E4, 4, 64), q_scale=T(F32, 4), rstd=T(F32, 4))),
        "rmsnorm_backward": (mp.rmsnorm_backward, dict(dy=T(BF, 4, 64), h=T(F32, 4, 64), gamma=T(F32, 64), rstd=T(F32, 4),
                                                       dx=T(F32, 4, 64), dh=T(F32, 4, 64), dgamma=T(F32, 64), workspace=ws)),
        "quantize_rows": (mp.quantize_rows, dict(x=T(BF, 4, 64), q=T(E4, 4, 64), scale=T(F32, 4))),
        "linear": (mp.linear, dict(x=T(E4, 4, 64), w=T(E4, 32, 64), y=T(BF, 4, 32), bias=T(BF, 32), residual=T(BF, 4, 32),
                                   z=T(BF, 4, 32), x_scale=T(F32, 4), w_scale=T(F32, 32), workspace=ws)),
        "linear_backward": (mp.linear_backward, dict(dz=T(BF, 4, 32), x=T(BF, 4, 64), w=T(BF, 32, 64), dx=T(BF, 4, 64),
                                                     z_prev=T(BF, 4, 64), dw=T(F32, 32, 64), dbias=T(F32, 32), workspace=ws)),
    }


@pytest.fixture
def recorded(monkeypatch):
    """Calls that would have reached the library, by name; nothing is launched."""
    reached = []

    class Library:
        def __getattr__(self, name):
            return lambda *args: reached.append(name) or 0
    mp.feedforward._load_torch()
    monkeypatch.setattr(mp, "lib", lambda: Library())
    monkeypatch.setattr(mp.feedforward, "_current_device", lambda: 0, raising=False)
    return reached


OPERANDS = [(f, a) for f, (_, args) in calls().items() for a in args]


@pytest.mark.parametrize("name", sorted(calls()))
def test_tensors_of_one_device_pass(recorded, name):
    f, args = calls()[name]
    f(**args, stream=0)
    assert len(recorded) == 1


@pytest.mark.parametrize("name,argument", OPERANDS)
@pytest.mark.parametrize("device", [1, -1])
def test_a_tensor_elsewhere_is_refused(recorded, name, argument, device):
    """One tensor, or the workspace, on another device or on the CPU."""
    f, args = calls()[name]
    args[argument]._device = device
    with pytest.raises(ValueError, match="cuda|CUDA"):
        f(**args, stream=0)
    assert not recorded


@pytest.mark.parametrize("name", sorted(calls()))
def test_a_device_that_is_not_current_is_refused(recorded, name):
    """All tensors on cuda:1 while cuda:0 is current: a launch would go to the
    current device's stream with the other one's addresses."""
    f, args = calls()[name]
    for t in args.values():
        t._device = 1
    with pytest.raises(ValueError, match="current"):
        f(**args, stream=0)
    assert not recorded


@pytest.mark.parametrize("name", ["rmsnorm_backward", "linear", "linear_backward"])
def test_a_workspace_with_gaps_is_refused(recorded, name):
    f, args = calls()[name]
    args["workspace"] = T(torch.uint8, 1 << 20, contiguous=False)
    with pytest.raises(ValueError, match="workspace"):
        f(**args, stream=0)
    assert not recorded


# ------------------------------------------------- derivatives without z --

def test_dx_through_an_activation_needs_its_argument():
    """act_prev names a derivative that is taken at z_prev: dx without z_prev
    is refused, not left without it.  Other outputs do not need z_prev."""
    fake = 1 << 20
    L = mp.lib()

    def status(**kw):
        a = mp.feedforward.OptLinearGradArgs(dz=fake, x=fake, w=fake, m=4, n=64, k=32, dz_ld=64, x_ld=32, w_ld=32, z_prev_ld=32,
                                             dx_ld=32)
        for name, v in kw.items():
            setattr(a, name, v)
        return L.opt_linear_backward(ctypes.byref(a), None, 0, None)      # no workspace: a call that is let through stops there
    for act in (1, 2, 3):
        assert status(dx=fake, act_prev=act) == mp.OPT_ERR_INVALID_ARG
        assert status(dx=fake, act_prev=act, z_prev=fake) == mp.OPT_ERR_WORKSPACE
        assert status(dw=fake, act_prev=act) == mp.OPT_ERR_WORKSPACE
    assert status(dx=fake) == status(dx=fake, z_prev=fake) == mp.OPT_ERR_WORKSPACE

"""What a call makes of a Branch's and a Dropout's fields, which may change between calls: it takes their tensors' addresses,
their sizes and the gate's rows as they are then.  The library is replaced by a recorder and tensors by stand-ins, so nothing
here needs a device or launches a kernel."""
import copy
import ctypes
import types

import pytest
import torch

W, M, N = 2, 8, 64


@pytest.fixture(scope="module")
def car():
    import __graft_entry__

    __graft_entry__.build()
    import rank_sum_reduce_gb300 as car

    return car


class Tensor:
    """As much of a CUDA tensor as the binding looks at."""

    def __init__(self, at, shape, dtype=torch.bfloat16, device=0):
        self.at, self.shape, self.dtype, self.dev = at, shape, dtype, device
        self.is_cuda, self.device = True, types.SimpleNamespace(index=device)

    def numel(self):
        return int(torch.Size(self.shape).numel())

    def element_size(self):
        return self.dtype.itemsize

    @property
    def nbytes(self):
        return self.numel() * self.element_size()

    def data_ptr(self):
        return self.at

    def get_device(self):
        return self.dev

    def is_contiguous(self):
        return True

    def is_floating_point(self):
        return self.dtype.is_floating_point

    def is_complex(self):
        return self.dtype.is_complex


@pytest.fixture
def calls(car, monkeypatch):
    """The struct and the outputs of every call that reaches the library."""
    seen = []

    def record(name, at):
        def call(*args):
            b = car.car_branch.from_buffer_copy(car.car_branch.from_address(args[at]))
            d = car.car_dropout.from_buffer_copy(b.dropout.contents) if b.dropout else None
            seen.append(types.SimpleNamespace(name=name, branch=b, dropout=d, args=args))
            return car.CAR_OK
        return call

    def dropout(*args):
        seen.append(types.SimpleNamespace(name="dropout", dropout=car.car_dropout.from_buffer_copy(car.car_dropout.from_address(args[2]))))
        return car.CAR_OK

    monkeypatch.setattr(car, "_lib", types.SimpleNamespace(
        car_reduce_branch_residual_rmsnorm=record("forward", 2), car_reduce_branch_residual_rmsnorm_backward=record("backward", 2),
        car_reduce_dropout=dropout, car_branch_workspace_bytes=lambda h, b: 0))
    return seen


def handle(car):
    c = object.__new__(car.Car)
    c.h, c.W, c.M, c.N, c.dtype, c.device = None, W, M, N, "bf16", 0
    c.D, c._row, c._branch_sizes, c._type = M * N * 2, N * 2, {}, torch.bfloat16
    return c


def forward(c, b, weight=None):
    t = [Tensor(0x1000 * (i + 1), (M, N)) for i in range(W + 3)]
    weight = weight or Tensor(0x100, (N,))
    c.reduce_branch_residual_rmsnorm(t[:W], b, t[W], weight, 1e-6, t[W + 1], t[W + 2], stream=0)


def backward(c, b, weight=None, dgate=None):
    t = [Tensor(0x1000 * (i + 1), (M, N)) for i in range(W + 3)]
    weight = weight or Tensor(0x100, (N,))
    c.reduce_branch_residual_rmsnorm_backward(t[:W], b, t[W], t[W + 1], weight, 1e-6, None, t[W + 2], dgate=dgate, stream=0)


def test_the_struct_is_the_c_one(car):
    assert ctypes.sizeof(car.car_branch) == 48 and ctypes.sizeof(car.car_dropout) == 32


@pytest.mark.parametrize("call", [forward, backward])
def test_every_field_may_be_set_anew(car, calls, call):
    c, drop = handle(car), car.Dropout(0.25, 5, 6)
    b = car.Branch(Tensor(0x200, (N,)), 1e-5, Tensor(0x300, (4, N)), gate_rows=4, residual_scale=0.5, dropout=drop)
    call(c, b)
    s = calls[-1].branch
    assert (s.norm_weight, s.gate, s.gate_rows, s.residual_scale) == (0x200, 0x300, 4, 0.5)
    assert (calls[-1].dropout.p, calls[-1].dropout.seed, calls[-1].dropout.offset) == (0.25, 5, 6)
    b.norm_weight, b.gate, b.gate_rows, b.residual_scale = Tensor(0x400, (N,)), Tensor(0x500, (M, N)), 0, 2.0
    b.norm_eps, b.dropout = 0.25, car.Dropout(0.5, 7, 8)
    assert (b.norm_eps, b.gate_rows, b.residual_scale, b.dropout.p) == (0.25, 0, 2.0, 0.5)
    call(c, b)
    s = calls[-1].branch
    assert (s.norm_weight, s.norm_eps, s.gate, s.gate_rows, s.residual_scale) == (0x400, 0.25, 0x500, 0, 2.0)
    assert (calls[-1].dropout.p, calls[-1].dropout.seed, calls[-1].dropout.offset) == (0.5, 7, 8)
    b.norm_weight = b.gate = b.dropout = None
    call(c, b)
    s = calls[-1].branch
    assert (s.norm_weight, s.gate, calls[-1].dropout) == (None, None, None)


@pytest.mark.parametrize("call", [forward, backward])
def test_a_tensor_that_moved_is_found(car, calls, call):
    """As after p.data = other, module.to() or a resized storage: the same object at another address."""
    c, w, g = handle(car), Tensor(0x200, (N,)), Tensor(0x300, (N,))
    b = car.Branch(w, 1e-5, g)
    call(c, b)
    w.at, g.at = 0x600, 0x700
    call(c, b)
    assert (calls[-1].branch.norm_weight, calls[-1].branch.gate) == (0x600, 0x700)


@pytest.mark.parametrize("name", ["norm_weight", "gate"])
@pytest.mark.parametrize("change", [dict(shape=(N - 8,)), dict(dev=1), dict(is_contiguous=lambda: False)],
                         ids=["smaller", "device", "strides"])
def test_a_tensor_that_became_unfit_is_refused(car, calls, name, change):
    """Each call looks at it anew."""
    c, t = handle(car), Tensor(0x200, (N,))
    b = car.Branch(**{name: t})
    forward(c, b)
    for k, v in change.items():
        setattr(t, k, v)
    t.device.index = t.dev
    for call in (forward, backward):
        with pytest.raises(ValueError, match=name):
            call(c, b)
    assert len(calls) == 1


def test_the_gates_gradient_has_the_rows_that_the_kernel_writes(car, calls):
    c, f32 = handle(car), torch.float32
    b = car.Branch(gate=Tensor(0x300, (N,)))
    backward(c, b, dgate=Tensor(0x800, (N,), f32))
    b.gate, b.gate_rows = Tensor(0x500, (4, N)), 4
    with pytest.raises(ValueError, match="dgate"):
        backward(c, b, dgate=Tensor(0x800, (1, N), f32))
    backward(c, b, dgate=Tensor(0x800, (4, N), f32))
    assert [k.branch.gate_rows for k in calls] == [1, 4]
    with pytest.raises(ValueError, match="gate_rows"):
        b.gate_rows = -1
    assert b.gate_rows == 4


def test_dropout_takes_new_fields(car, calls, monkeypatch):
    c = handle(car)
    t = [Tensor(0x1000 * (i + 1), (M, N)) for i in range(W + 1)]
    step = Tensor(0x40, (1,), torch.int64)
    d = car.Dropout(0.5, 1, 2, offset_dev=step)
    c.reduce_dropout(t[:W], d, t[W], stream=0)
    assert (calls[-1].dropout.p, calls[-1].dropout.offset_dev) == (0.5, 0x40)
    step.at, d.p = 0x80, 0.25
    c.reduce_dropout(t[:W], d, t[W], stream=0)
    forward(c, car.Branch(dropout=d))
    assert [(k.dropout.p, k.dropout.offset_dev) for k in calls[1:]] == [(0.25, 0x80)] * 2
    for bad in (-0.1, 1.5, float("nan")):
        with pytest.raises(ValueError, match="p: "):
            d.p = bad
    with pytest.raises(ValueError, match="offset_dev: torch.int32"):
        d.offset_dev = Tensor(0x40, (1,), torch.int32)
    assert d.p == 0.25 and d.offset_dev is step
    d.offset_dev = None
    c.reduce_dropout(t[:W], d, t[W], stream=0)
    assert calls[-1].dropout.offset_dev is None


def test_two_branches_share_a_dropout(car, calls):
    """What is set on it holds for both, as before."""
    c, d = handle(car), car.Dropout(0.5, 1, 2)
    bs = [car.Branch(dropout=d), car.Branch(residual_scale=0.5, dropout=d)]
    d.seed, d.offset = 9, 2**64 + 10
    for b in bs:
        forward(c, b)
    assert [(k.dropout.seed, k.dropout.offset) for k in calls] == [(9, 10)] * 2


@pytest.mark.parametrize("call", [forward, backward])
@pytest.mark.parametrize("name", ["norm_weight", "gate", "weight"])
@pytest.mark.parametrize("bad", [torch.float32, torch.float64, torch.float16, torch.float8_e4m3fn, torch.complex64])
def test_weights_and_gates_of_another_type_are_refused(car, calls, call, name, bad):
    """Large enough all the same: an fp32 weight holds a bf16 one's bytes twice."""
    t = Tensor(0x300, (4 * N,) if bad.itemsize == 1 else (N,), bad)
    with pytest.raises(ValueError, match=f"{name}: {bad}"):
        call(handle(car), car.Branch(**({name: t} if name != "weight" else {})), **({} if name != "weight" else {name: t}))
    assert not calls


@pytest.mark.parametrize("call", [forward, backward])
@pytest.mark.parametrize("name,gate_rows,shape", [("gate", 1, (M, N)), ("gate", 1, (2, N)), ("gate", 4, (M, N)), ("gate", 2, (1, N)),
                                                  ("gate", 0, (M + 1, N)), ("norm_weight", 1, (M, N)), ("norm_weight", 1, (N + 8,)),
                                                  ("norm_weight", 1, (0,))])
def test_weights_and_gates_of_another_size_are_refused(car, calls, call, name, gate_rows, shape):
    """A gate of a row for every row is not a gate of all rows, whatever its first row holds."""
    with pytest.raises(ValueError, match=name):
        call(handle(car), car.Branch(gate_rows=gate_rows, **{name: Tensor(0x300, shape)}))
    assert not calls


@pytest.mark.parametrize("call", [forward, backward])
@pytest.mark.parametrize("gate_rows,shape", [(1, (N,)), (1, (1, N)), (4, (4, N)), (4, (4, 1, N)), (4, (4 * N,)), (0, (M, N)),
                                             (0, (2, M // 2, N)), (M, (M, N))])
def test_every_shape_of_as_many_values_is_taken(car, calls, call, gate_rows, shape):
    call(handle(car), car.Branch(gate=Tensor(0x300, shape), gate_rows=gate_rows))
    raw = Tensor(0x300, (torch.Size(shape).numel() * 2,), torch.uint8)     # the same as bytes
    call(handle(car), car.Branch(gate=raw, gate_rows=gate_rows, norm_weight=Tensor(0x200, (N,), torch.int16)))
    assert [k.branch.gate for k in calls] == [0x300] * 2


@pytest.mark.parametrize("bad", [torch.float32, torch.float16, torch.float64])
def test_a_gradient_of_another_type_for_a_gate_of_each_rows_own_is_refused(car, calls, bad):
    c, b = handle(car), car.Branch(gate=Tensor(0x300, (M, N)), gate_rows=0)
    with pytest.raises(ValueError, match=f"dgate: {bad}"):
        backward(c, b, dgate=Tensor(0x800, (M, N), bad))
    assert not calls
    backward(c, b, dgate=Tensor(0x800, (M, N)))
    assert len(calls) == 1


def test_copies_have_fields_of_their_own(car, calls):
    """What is set on a copy does not reach the first one's calls: not its number of gate rows either, by which its gradient
    is sized."""
    c, d = handle(car), car.Dropout(0.5, 1, 2)
    b = car.Branch(Tensor(0x200, (N,)), 1e-5, Tensor(0x300, (N,)), residual_scale=0.5, dropout=d)
    other, e = copy.copy(b), copy.copy(d)
    other.gate, other.gate_rows, other.residual_scale, other.norm_eps = Tensor(0x500, (4, N)), 4, 2.0, 0.25
    other.dropout, e.seed, e.p = None, 9, 0.25
    backward(c, b, dgate=Tensor(0x800, (N,), torch.float32))
    s = calls[-1].branch
    assert (s.norm_weight, s.gate, s.gate_rows, s.residual_scale, calls[-1].dropout.seed) == (0x200, 0x300, 1, 0.5, 1)
    assert abs(s.norm_eps - 1e-5) < 1e-11 and (d.seed, d.p) == (1, 0.5) and (e.seed, e.offset, e.p) == (9, 2, 0.25)
    backward(c, other, dgate=Tensor(0x800, (4, N), torch.float32))
    s = calls[-1].branch
    assert (s.norm_weight, s.gate, s.gate_rows, s.residual_scale, calls[-1].dropout) == (0x200, 0x500, 4, 2.0, None)
    for x in (b, d):
        with pytest.raises(ValueError):   # addresses are this process's
            copy.deepcopy(x)


def test_the_struct_is_ready_for_the_c_calls(car):
    """Without a call through a handle: what was given and what was set."""
    d = car.Dropout(0.5, 1, 2, offset_dev=Tensor(0x40, (1,), torch.int64))
    b = car.Branch(Tensor(0x200, (N,)), 1e-5, Tensor(0x300, (4, N)), 4, 0.5, d)
    s = car.car_branch.from_address(b.address)
    assert (s.norm_weight, s.gate, s.gate_rows, s.residual_scale) == (0x200, 0x300, 4, 0.5)
    assert s.dropout.contents.offset_dev == 0x40 and ctypes.addressof(b.ref._obj) == b.address
    b.norm_weight, b.gate = None, Tensor(0x500, (4, N))
    assert (s.norm_weight, s.gate) == (None, 0x500)

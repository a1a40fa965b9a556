"""The grouped products' gradients on small whole numbers, whose fp32 sums are
exact in any order: equality, so that one lost, doubled or foreign row shows
at any length of a sum.  dy holds -1, 0 and 1 (a quarter of it not 0), x and w
hold -1 and 1: a row that is left out moves a quarter of its expert's
gradients by 1, and sums of up to 2^24 rows are exact.  bf16 results are the
exact ones, rounded once.  Rows that are not live hold NaN.

The reference products run in fp32 on the GPU, exact for the same reason."""

import pytest

torch = pytest.importorskip("torch")

import expanded_dispatch_layout_amd as M  # noqa: E402

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

BF = torch.bfloat16


def signs(shape, gen):
    return torch.randint(0, 2, shape, generator=gen, device="cuda", dtype=torch.int8).mul_(
        2).sub_(1).to(BF)


class Data:
    """Experts of `counts` rows in a buffer of `capacity` rows."""

    def __init__(self, counts, n, k, align, capacity, seed=0):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed + n + k)
        self.n, self.k, self.align, self.E = n, k, align, len(counts)
        self.dy = signs((capacity, n), gen)
        self.dy.masked_fill_(torch.rand((capacity, n), generator=gen, device="cuda") >= 0.25, 0)
        self.x, self.w = signs((capacity, k), gen), signs((self.E, n, k), gen)
        self.live, end = [], 0
        for c in counts:
            self.live.append(slice(end, end + c))
            end = -(-(end + c) // align) * align
        assert end <= capacity
        dead = torch.ones(capacity, dtype=torch.bool, device="cuda")
        for s in self.live:
            dead[s] = False
        self.dead = dead
        self.dy[dead], self.x[dead] = float("nan"), float("nan")
        ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        self.psum, self.status = ints([s.stop for s in self.live]), ints([end, 0])

    def sums(self, e):
        """Expert e's weight gradient in fp32, 32768 rows at a time."""
        out = torch.zeros((self.n, self.k), device="cuda")
        for first in range(self.live[e].start, self.live[e].stop, 32768):
            rows = slice(first, min(first + 32768, self.live[e].stop))
            out += self.dy[rows].float().t().contiguous() @ self.x[rows].float()
        return out

    def wgrad(self, f32, accumulate):
        dw = torch.full((self.E, self.n, self.k), 5.0 if accumulate else float("nan"),
                        dtype=torch.float32 if f32 else BF, device="cuda")
        need = M.moe_grouped_wgrad_workspace_bytes(self.dy.shape[0], self.n, self.k, self.E)
        ws = torch.full((need,), 0xff, dtype=torch.uint8, device="cuda") if need else None
        M.moe_grouped_wgrad_bf16(self.dy, self.x, self.psum, self.status, self.align, dw, ws,
                                 accumulate=accumulate)
        for e in range(self.E):
            want = self.sums(e) + (5.0 if accumulate else 0.0)
            assert torch.equal(dw[e], want.to(dw.dtype)), f"dw[{e}] f32 {f32} added {accumulate}"

    def dgrad(self):
        dx = torch.full((self.dy.shape[0], self.k), 7.0, dtype=BF, device="cuda")
        M.moe_grouped_dgrad_bf16(self.dy, self.w, self.psum, self.status, self.align, dx)
        assert torch.all(dx[self.dead] == 7.0)
        for e, s in enumerate(self.live):
            want = self.dy[s].float() @ self.w[e].float()
            assert torch.equal(dx[s], want.to(BF)), f"dx of expert {e}"


def tight(counts, align):
    return sum(-(-c // align) * align for c in counts) + align


SUMS = [
    ([1], 128, 64, 16),
    ([31, 0, 32, 33, 64, 1], 256, 192, 16),
    ([3000], 256, 256, 128),
    ([5000, 1], 128, 128, 16),
    ([20000, 1], 128, 128, 16),                    # parts
    ([9000, 0, 4500, 8200], 256, 320, 16),
    ([70, 0, 16000, 1, 9000], 128, 64, 128),
    ([12001, 11000], 384, 576, 64),
    ([200000], 128, 128, 16),
    ([65] * 8, 2048, 1024, 16),                    # 64 x 64, 128 x 128 and 256 x 256 tiles
    ([2000, 0, 300, 2300], 256, 4160, 64),
    ([700, 1, 0, 6001, 33, 2048, 97, 512], 2048, 1088, 32),
    ([40, 0, 1, 70] * 16, 384, 320, 16),
]


@pytest.mark.parametrize("counts,n,k,align", SUMS, ids=lambda v: str(v).replace(" ", "")[:24])
def test_whole_numbers(counts, n, k, align):
    print(f"{counts[:8]} n {n} k {k} align {align}", flush=True)
    d = Data(counts, n, k, align, tight(counts, align))
    d.dgrad()
    for f32 in (True, False):
        for accumulate in (False, True):
            d.wgrad(f32, accumulate)


# Rows received, topk, live rows per expert (8 of 256 experts are here), n, k, align: the
# layer classes' own buffers hold topk rows for each row received, most of them unused.
OWN = [
    (512, 8, [16, 9, 20, 0, 31, 17, 12, 23], 2048, 1024, 128),
    (4096, 8, [128, 100, 157, 131, 0, 201, 140, 167], 2048, 1024, 128),
    (4096, 8, [128, 100, 157, 131, 0, 201, 140, 167], 1024, 1024, 128),
    (4096, 8, [0, 0, 0, 0, 0, 0, 0, 1], 1024, 1024, 128),
    (4096, 8, [0] * 8, 256, 192, 16),
    (1024, 8, [1, 0, 260, 3, 64, 65, 63, 500], 4096, 512, 64),
    (8192, 8, [40, 30, 1, 0], 512, 256, 16),
    (2000, 32, [77], 1024, 320, 32),
]


@pytest.mark.parametrize("rows,topk,counts,n,k,align", OWN, ids=[
    f"{c[0]}x{c[1]}-{sum(c[2])}-n{c[3]}-k{c[4]}" for c in OWN])
def test_buffers_of_the_layers_own_capacity(rows, topk, counts, n, k, align):
    """Far more rows of capacity than live ones, in buffers as TrainableBf16MoE
    allocates them."""
    print(f"rows {rows} topk {topk} {counts} n {n} k {k} align {align}", flush=True)
    cap = M.moe_expand_capacity(rows, topk, len(counts), align)
    assert cap >= 4 * sum(counts)
    d = Data(counts, n, k, align, cap, seed=1)
    d.dgrad()
    d.wgrad(True, False)
    d.wgrad(True, True)
    d.wgrad(False, False)


@pytest.mark.slow
def test_a_long_sum_past_32_bits():
    """300001 rows of 8192 columns (element offsets past 2^31), and 77 behind them."""
    d = Data([300001, 77], 8192, 128, 32, 300032 + 128)
    print("dgrad", flush=True)
    d.dgrad()
    print("wgrad", flush=True)
    d.wgrad(True, False)
    d.wgrad(False, True)

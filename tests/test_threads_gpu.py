"""The operators around the attention from several host threads at once, each on a stream and with tensors of
its own: the results of the same calls made one after the other, bit for bit."""
import threading

import pytest
import torch

from causal_attention_attn_b200 import attn, build
from tests import rows_reference as ref

pytestmark = pytest.mark.gpu
D, PAGE, PER = 128, 16, 4


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    if torch.cuda.get_device_capability(0) != (10, 0):
        pytest.skip("needs an sm_100 device")
    build.build()
    attn.load_library()
    yield
    torch.cuda.synchronize()
    assert attn.device_status() == 0


class Layer:
    """One thread's tensors, and a step through every operator."""

    def __init__(self, seed, B, Hq, Hkv, S):
        g = torch.Generator().manual_seed(seed)
        draw = lambda *shape: torch.randn(shape, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
        self.q, self.k, self.v, self.dq, self.dk = (draw(B, H, S, D) for H in (Hq, Hkv, Hkv, Hq, Hkv))
        self.w = [draw(D) for _ in range(2)]
        self.cos, self.sin = (t.cuda() for t in ref.angle_tables(PAGE * PER, D))
        n = B * PER + 6
        self.pages = [draw(n, Hkv, PAGE, D) for _ in range(2)]
        self.codes = [torch.randint(0, 120, (n, Hkv, PAGE, D), generator=g).to(torch.uint8).cuda() for _ in range(2)]
        self.coef = torch.full((Hkv, D), 2.0 ** -5).cuda()
        self.table = torch.arange(B * PER, dtype=torch.int32).view(B, PER).cuda()
        self.ptab = torch.arange(B * PER, n, dtype=torch.int32).cuda()
        self.plen = torch.tensor([6 * PAGE - 3], dtype=torch.int32).cuda()
        self.lens = torch.full((B,), S, dtype=torch.int32).cuda()

    def step(self):
        kw = dict(q_weight=self.w[0], k_weight=self.w[1])
        qr, kr = attn.attn_qk_norm_rope(self.q, self.k, self.cos, self.sin, **kw)
        back = attn.attn_qk_norm_rope_bwd(self.q, self.k, self.cos, self.sin, self.dq, self.dk, **kw)
        qo = attn.attn_append_paged(self.k, self.v, self.cos, self.sin, *self.pages, self.table, self.lens, q=self.q, **kw)
        attn.attn_append_paged_fp8(self.k, self.v, self.cos, self.sin, *self.codes, self.coef, self.coef, self.table,
                                   self.lens, k_weight=self.w[1])
        last = qo[:, :, -1:].contiguous()
        cap = PAGE * PER
        near = attn.attn_decode_prefix(last, *self.pages, self.ptab, self.plen, self.table, self.lens, 6 * PAGE, cap)
        far = attn.attn_decode_prefix(last, *self.pages, self.ptab, self.plen, self.table, self.lens, 6 * PAGE, cap,
                                      scale=0.05)
        return [qr, kr, *back, qo, *self.pages, *self.codes, *near, *far]


def test_four_threads():
    layers = [Layer(i, B=1 + i, Hq=(32, 8, 40, 6)[i], Hkv=(8, 2, 2, 6)[i], S=17 + 10 * i) for i in range(4)]
    want = [[t.clone() for t in layer.step()] for layer in layers]
    torch.cuda.synchronize()
    wrong, start = [], threading.Barrier(len(layers))

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                start.wait(60)
                for n in range(40):
                    got = layers[i].step()
                    if n % 8 == 7:
                        torch.cuda.current_stream().synchronize()
                        if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                            wrong.append((i, n))
        except BaseException as e:  # noqa: BLE001
            wrong.append((i, repr(e)))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(layers))]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
    torch.cuda.synchronize()
    assert not wrong and not any(t.is_alive() for t in threads)

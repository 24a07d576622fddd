"""A message between the CTAs of a cluster that is held back (opt_selftest_mail): the waits
for it run out, every message that came in full is right, everything behind is NaN,
and the context goes on.  Sums of small whole numbers: exact in fp32."""

import time

import pytest

from gpu_helpers import require_gpu, torch
import mixed_precision_optimizer_gb300 as mp

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def expected(ctas, messages):
    k, t = torch.arange(messages).view(1, -1, 1), torch.arange(64).view(1, 1, -1)
    one = 1000 * k * ctas + 64 * (ctas * (ctas - 1) // 2) + ctas * t
    return one.expand(ctas, messages, 64).float().cuda()


@pytest.mark.parametrize("ctas", [2, 3, 8])
@pytest.mark.parametrize("messages", [1, 2, 17, 64])
def test_all_messages_come(ctas, messages):
    sums = torch.zeros(ctas, messages, 64, device="cuda")
    mp.selftest_mail(sums)
    assert torch.equal(sums, expected(ctas, messages))


@pytest.mark.parametrize("ctas", [2, 3, 8])
@pytest.mark.parametrize("held_back", [0, 1, 2, 6])
def test_a_message_held_back(ctas, held_back):
    messages = 7
    sums, want = torch.zeros(ctas, messages, 64, device="cuda"), expected(ctas, messages)
    torch.cuda.synchronize()
    t0 = time.monotonic()
    mp.selftest_mail(sums, held_back)
    torch.cuda.synchronize()
    assert 0.15 < time.monotonic() - t0 < 30            # two or three waits of 0.2 s; nothing hangs
    want[0, held_back:] = float("nan")
    want[1:, held_back + 1:] = float("nan")
    assert torch.equal(sums.isnan(), want.isnan()) and torch.equal(sums.nan_to_num(), want.nan_to_num())
    # and a cluster's kernel right behind it is whole
    x, labels = torch.zeros(4, 40000, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda")
    lse = torch.zeros(4, device="cuda")
    mp.cross_entropy(x, labels, lse=lse)
    assert bool((lse - 10.596634733).abs().max() < 1e-5)          # log 40000


def test_refusals():
    sums = torch.zeros(2, 4, 64, device="cuda")
    for bad in (torch.zeros(1, 4, 64, device="cuda"), torch.zeros(9, 4, 64, device="cuda"), torch.zeros(2, 65, 64, device="cuda")):
        with pytest.raises(mp.MpoptError, match="INVALID"):
            mp.selftest_mail(bad)
    for k in (-2, 4):
        with pytest.raises(mp.MpoptError, match="INVALID"):
            mp.selftest_mail(sums, k)
    with pytest.raises(ValueError, match="sums has shape"):
        mp.selftest_mail(torch.zeros(2, 4, 63, device="cuda"))
    with pytest.raises(TypeError, match="sums must be"):
        mp.selftest_mail(sums.double())

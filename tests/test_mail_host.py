"""The messages between the CTAs of a cluster without a GPU: the rule of csrc/mail.h, which
the recurrence's and the cross-entropy's kernels follow, over a model of the mbarriers
(mail_model.cpp).  Whatever is late, nobody takes one message for another, everybody
ends, and after a loss nobody receives a later message."""

import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
GXX = shutil.which("g++")
pytestmark = pytest.mark.skipif(GXX is None, reason="needs g++")


def program(tmp_path_factory, name, *flags):
    exe = str(tmp_path_factory.mktemp("mail") / name)
    r = subprocess.run([GXX, "-std=c++20", "-O1", "-pthread", *flags, os.path.join(HERE, "mail_model.cpp"), "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return exe


@pytest.fixture(scope="module")
def model(tmp_path_factory):
    return program(tmp_path_factory, "model")


def run(exe, *args):
    r = subprocess.run([exe, *map(str, args)], capture_output=True, text=True, timeout=100)
    return r.returncode, r.stdout


@pytest.mark.parametrize("ctas,threads", [(2, 1), (3, 2), (8, 2)])
def test_all_messages_come(model, ctas, threads):
    code, out = run(model, ctas, threads, 200, 60000, -1, 0, 0)
    assert code == 0 and out.split() == ["200"] * (ctas * threads)


@pytest.mark.parametrize("ctas,threads", [(2, 1), (2, 3), (3, 1), (8, 2)])
@pytest.mark.parametrize("message", [0, 1, 3, 7])
def test_a_late_part(model, ctas, threads, message):
    """A part that comes to a message when others have given up on it: those have lost it, it
    may receive it, and nobody the next."""
    code, out = run(model, ctas, threads, 8, 100, ctas - 1, message, 0)
    assert code == 0, out
    came = [int(v) for v in out.split()]
    assert min(came) <= message and max(came) <= message + 1


@pytest.mark.parametrize("ctas,threads", [(2, 1), (3, 2)])
def test_late_mail_finds_its_cta(model, ctas, threads):
    """The last message to CTA 0 arrives behind the kernel's last barrier: CTA 0 is still there."""
    code, out = run(model, ctas, threads, 4, 100, ctas - 1, 3, 1)
    assert code == 0, out
    came = [int(v) for v in out.split()]
    assert came[:threads] == [3] * threads and came[threads:] == [4] * (len(came) - threads)


def test_the_model_sees_a_part_that_goes_on_sending(tmp_path_factory):
    """The same model over the rule that a part which lost a message sends the later ones:
    a late part then takes message 2 for message 0."""
    exe = program(tmp_path_factory, "planted", "-DPLANTED")
    code, out = run(exe, 2, 1, 4, 100, 1, 0, 0)
    assert code == 1 and "took message" in out


def test_selftest_refuses_host_memory():
    torch = pytest.importorskip("torch")
    import mixed_precision_optimizer_gb300 as mp
    with pytest.raises(ValueError, match="CUDA"):
        mp.selftest_mail(torch.zeros(2, 4, 64))


def test_selftest_refusals():
    pytest.importorskip("torch")
    import mixed_precision_optimizer_gb300 as mp
    from mixed_precision_optimizer_gb300 import build_lib
    build_lib.build()
    call, fake = mp.lib().opt_selftest_mail, 1 << 20
    for ctas, messages, held in ((1, 4, -1), (9, 4, -1), (2, 0, -1), (2, 65, -1), (2, 4, -2), (2, 4, 4)):
        assert call(fake, ctas, messages, held, None) == 1
    assert call(None, 2, 4, -1, None) == 1 and call(fake + 2, 2, 4, -1, None) == 3

"""The shares of the rows' own tokens beside shared ones (kv_share), by a kernel of its own: whatever SMs the CTAs are put
on and in whatever order they come, each share is one CTA's."""
import ctypes
import os
import subprocess

import pytest
import torch

from prefill_dsa_indexer_gb300 import build

pytestmark = pytest.mark.gpu

OWN_SMS = 256
LINGER = 40000  # cycles of a share, some 20 us


@pytest.fixture(scope="module")
def launch(tmp_path_factory):
    lib = str(tmp_path_factory.mktemp("shares") / "shares.so")
    source = os.path.join(os.path.dirname(os.path.abspath(__file__)), "kv_shares.cu")
    subprocess.run([build.nvcc(), *build.ARCH, *build.FLAGS, f"-I{build.CSRC}", "-shared", source, "-o", lib], check=True)
    fn = ctypes.CDLL(lib).shares_launch
    fn.argtypes = [ctypes.c_void_p] * 3 + [ctypes.c_int32] * 3 + [ctypes.c_void_p]

    def run(sms, ctas, smem, taken=()):
        """Shares of each CTA and how often each was taken; taken: (SM, how many of its shares are gone already)."""
        own = torch.zeros(1 + OWN_SMS, dtype=torch.int32, device="cuda")
        own[0] = sms
        for sm, n in taken:
            own[1 + sm] = n
        made, by = torch.zeros(ctas, dtype=torch.int32, device="cuda"), torch.full((ctas,), -7, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        assert fn(own.data_ptr(), made.data_ptr(), by.data_ptr(), LINGER, ctas, smem,
                  torch.cuda.current_stream().cuda_stream) == 0
        return by, made
    return run


def sm_count():
    return torch.cuda.get_device_properties(0).multi_processor_count


# two CTAs an SM, as the attention kernels have; one, so that the others come late and to whatever SM is free; many
@pytest.mark.parametrize("smem", [100 << 10, 200 << 10, 1 << 10])
@pytest.mark.parametrize("sms", [1, 4, 8, 56, 75, 120, 148])
def test_each_share_is_one_ctas(launch, smem, sms):
    most = 2 * sm_count()
    for ctas in sorted({most, 2 * sms + 1, min(most, 2 * sms + 57)}):
        for _ in range(5):
            by, made = launch(sms, ctas, smem)
            assert made.tolist() == [1] * (2 * sms) + [0] * (ctas - 2 * sms), (ctas, made.tolist())
            taken = by[by >= 0].tolist()
            assert (by >= -1).all() and sorted(taken) == list(range(2 * sms))


@pytest.mark.parametrize("smem", [100 << 10, 200 << 10])
def test_shares_that_others_took(launch, smem):
    """Shares that are gone when the CTAs come (late ones of other SMs took them) are nobody's here, and the others'
    still one CTA's each."""
    for sms, gone in ((56, [(0, 2), (17, 1), (55, 2)]), (8, [(i, 2) for i in range(8)]), (20, [(3, 1), (4, 5)])):
        by, made = launch(sms, 2 * sm_count(), smem, gone)
        want = [1] * (2 * sms)
        for sm, n in gone:
            want[2 * sm:2 * sm + min(n, 2)] = [0] * min(n, 2)
        assert made[:2 * sms].tolist() == want and (made[2 * sms:] == 0).all() and (by >= -1).all()


def test_all_sms_are_the_grid_as_it_is(launch):
    """Where the own tokens get every SM a CTA's share is its number."""
    n = sm_count()
    for sms, ctas in ((n, 2 * n), (n + 1, 2 * n), (8, 16), (8, 5)):
        by, made = launch(sms, ctas, 100 << 10)
        assert by.tolist() == list(range(ctas)) and (made == 1).all()


def test_shares_beside_a_kernel_that_holds_sms(launch):
    """CTAs that find no room come when others have left."""
    a, stream = torch.randn(2048, 2048, device="cuda", dtype=torch.bfloat16), torch.cuda.Stream()
    for i in range(20):
        with torch.cuda.stream(stream):
            for _ in range(1 + i % 4):
                a @ a
        by, made = launch(56, 2 * sm_count(), 100 << 10)
        assert made.tolist() == [1] * 112 + [0] * (2 * sm_count() - 112)
    torch.cuda.synchronize()

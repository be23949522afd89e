"""Grids of the paged-cache kernels follow the device, not a number of SMs written down.  Host-only."""
import re

from tests import pages_plan


def test_no_launch_names_a_number_of_sms():
    for name in ("pages.cu", "pages_api.cu", "attn_pages.cu", "attn_pages_f32.cu", "attn_pages_16.cu"):
        with open(f"{pages_plan.CSRC}/{name}") as f:
            code = re.sub(r"//[^\n]*", "", f.read())
        assert not re.search(r"\b(148|152)\b", code), name

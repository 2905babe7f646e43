"""The binding's module-level paths, without a GPU."""
import os

import attention_attn_fwd_bwd_gb300 as af


def test_the_package_folder_keeps_its_name():
    assert os.path.samefile(af._HERE, os.path.dirname(af.__file__))
    assert os.path.dirname(os.path.dirname(af.library_path())) == af._HERE

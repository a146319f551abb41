"""What the package offers after a plain import."""
import subprocess
import sys

import pytest


@pytest.mark.parametrize("name", ["q8.decode_shared", "q8.Cache", "binding.decode", "decode", "workloads"])
def test_attributes_after_a_plain_import(name):
    """In a process of its own: another test may have imported the module already."""
    code = ("import sys, grouped_query_attention_mqa_b200 as m\n"
            "assert m.__name__ + '.q8' not in sys.modules\n"
            f"m.{name}")
    subprocess.run([sys.executable, "-c", code], check=True)


def test_unknown_attributes_are_refused():
    import grouped_query_attention_mqa_b200 as m
    with pytest.raises(AttributeError):
        m.q9

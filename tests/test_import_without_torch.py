"""The C names in a process that has no torch: addresses and a stream of the
caller's own, as before the losses came (CPU)."""

import subprocess
import sys

from conftest import ROOT

HIDE = "import sys\nsys.modules['torch'] = None        # import torch raises ModuleNotFoundError\n"


def _run(code):
    return subprocess.run([sys.executable, "-c", HIDE + code], capture_output=True, text=True, cwd=ROOT, timeout=300)


def test_the_c_names_need_no_torch():
    res = _run("import context_packed_sequence_amd as thd\n"
               "assert 'vocabulary' in thd.thd_strerror(thd.THD_ERR_LABEL)\n"
               "assert thd.thd_pack_workspace_bytes(4, 128) > 0\n"
               "assert thd.thd_loss_workspace_bytes(2, 131072, thd.THD_BF16, 1) > 0\n"
               "try:\n"
               "    thd.thd_policy_loss(4096, thd.THD_BF16, -1, 8, 8, 4096, None, 4096, None, 4096, None, .2, .2, 0.,\n"
               "                        4096, 4096, 4096, 8, None, None, 0, stream=0)\n"
               "except thd.ThdError as e:\n"
               "    print(e.code)\n"
               "print(hasattr(thd, 'Route'), hasattr(thd, 'policy_loss'))\n")
    assert res.returncode == 0, res.stderr
    assert res.stdout.split() == ["-1", "True", "False"]


def test_a_broken_torch_is_reported():
    # only its absence is taken for a process without torch
    code = ("class Broken:\n"
            "    def find_spec(self, name, path=None, target=None):\n"
            "        if name == 'torch':\n"
            "            raise ImportError('half installed')\n"
            "del sys.modules['torch']\n"
            "sys.meta_path.insert(0, Broken())\n"
            "import context_packed_sequence_amd\n")
    res = _run(code)
    assert res.returncode != 0 and "half installed" in res.stderr

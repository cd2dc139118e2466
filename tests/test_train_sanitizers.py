"""The training-side C-ABI layer under AddressSanitizer and
UndefinedBehaviorSanitizer (CPU): 4000 random GroupNorm shapes and gradient
lists through tests/sanitize/train_driver.cpp, whose stand-in launchers check
the plans against what the kernels assume."""
from test_sanitizers import _build_and_run


def test_train_c_abi_layer_under_sanitizers(tmp_path):
    _build_and_run(tmp_path, "g++",
                   ["tests/sanitize/train_driver.cpp",
                    "convolution_video_vae_amd/csrc/conv3d_train_api.cpp"],
                   ["-std=c++17", "-Wall"], "train_driver", "train driver ok")

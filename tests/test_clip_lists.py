"""Long gradient lists through the C-ABI layer, under AddressSanitizer and
UndefinedBehaviorSanitizer (CPU, tests/sanitize/clip_driver.cpp)."""
from test_sanitizers import _build_and_run


def test_clip_work_grows_with_the_list(tmp_path):
    _build_and_run(tmp_path, "g++",
                   ["tests/sanitize/clip_driver.cpp",
                    "convolution_video_vae_amd/csrc/conv3d_train_api.cpp"],
                   ["-std=c++17", "-Wall"], "clip_driver", "clip driver ok")

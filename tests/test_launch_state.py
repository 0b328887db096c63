"""Launch code keeps nothing of a device between calls: an SM count is asked of the current device
(two devices, or two threads at their first call, must not share it)."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "paged_fp8_kv_append_gb300", "csrc")


def test_sm_count_is_asked_of_the_current_device():
    asked = 0
    for name in sorted(os.listdir(CSRC)):
        with open(os.path.join(CSRC, name)) as f:
            text = f.read()
        for call in re.findall(r"cudaDeviceGetAttribute\(([^;]*?)\)\s*[!=;]", text):
            args = [a.strip() for a in call.split(",")]
            if args[1] == "cudaDevAttrMultiProcessorCount":
                assert args[2] != "0", f"{name}: the SM count of device 0, whichever is current"
                asked += 1
        assert not re.search(r"static\s+int\s+sms\b", text), f"{name}: an SM count kept between calls"
    assert asked == 1, "one helper asks"

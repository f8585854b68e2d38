"""How the timeouts of the 8-bit product are reported (host logic, no GPU): kernels on other streams add to the
device's count while a status call reads it, and none of theirs may be lost.  The device is a counter here; what
other streams do between a call's read and its report is a function run there."""
import os
import re
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "lut_dequant_gemv_b200", "csrc")

PROGRAM = r"""
#include "timeouts.cuh"
#include <cstdio>
#include <functional>
#include <thread>
#include <vector>

static std::atomic<uint32_t> device_count{0};
static bool status_call(sqz::ReportedTimeouts& r, const std::function<void()>& meanwhile = [] {}) {
    const uint32_t read = device_count.load();
    meanwhile();
    return r.take(read);
}
#define EXPECT(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return 1; } } while (0)

int main() {
    const auto timeout = [] { ++device_count; };
    {
        sqz::ReportedTimeouts r;
        EXPECT(!status_call(r));
        timeout();
        EXPECT(status_call(r));
        EXPECT(!status_call(r));             // once
        EXPECT(!status_call(r, timeout));    // after this call's read ...
        EXPECT(status_call(r));              // ... is the next one's
        timeout();
        EXPECT(status_call(r, timeout));     // one before the read, one after
        EXPECT(status_call(r));
        EXPECT(!status_call(r));
        timeout();                           // a call inside another: the later read reports both
        bool inner = false;
        const bool outer = status_call(r, [&] { timeout(); inner = status_call(r); });
        EXPECT(inner && !outer);
        EXPECT(!status_call(r));
    }
    {  // the count wraps
        device_count = 0;
        sqz::ReportedTimeouts r;
        for (uint32_t c : {0x7fffffffu, 0xfffffff0u, 5u}) {
            device_count = c;
            EXPECT(status_call(r) && !status_call(r));
        }
    }
    {  // callers and timeouts at once: whatever is left over is reported at the end, and then nothing is
        device_count = 0;
        sqz::ReportedTimeouts r;
        std::atomic<int> reports{0};
        std::vector<std::thread> threads;
        for (int t = 0; t < 4; ++t)
            threads.emplace_back([&, t] {
                for (int i = 0; i < 20000; ++i) {
                    if (t < 2) ++device_count;
                    else reports += status_call(r);
                }
            });
        for (auto& t : threads) t.join();
        ++device_count;
        EXPECT(status_call(r) && !status_call(r));
        EXPECT(reports.load() <= 40000);
    }
    return 0;
}
"""


def test_every_timeout_is_reported_once(tmp_path):
    src, exe = tmp_path / "timeouts.cpp", tmp_path / "timeouts"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-I", CSRC, "-x", "c++", str(src), "-o", str(exe)], check=True)
    done = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert done.returncode == 0, done.stdout


def test_the_status_call_reads_and_never_writes_the_count():
    """A clear behind the read would be on the caller's stream only."""
    text = open(os.path.join(CSRC, "sqz_fp8.cu")).read()
    body = text[text.index("sqz_status sqz_fp8_status("):]
    assert ".take(" in body and not re.search(r"cudaMemset|HostToDevice|<<<|cudaLaunch", body)
    kernels = open(os.path.join(CSRC, "kernels_fp8.cuh")).read()
    assert len(re.findall(r"atomicAdd\(p\.status, 1u?\)", kernels)) == 2 and "atomicOr" not in kernels

"""Host threads that share a stream's workspace, without a GPU: the bookkeeping of
csrc/workspace.h under several threads."""
import os
import subprocess

from attn_fwd_04_b200 import build as fa_build

HARNESS = r"""
#include "workspace.h"

#include <atomic>
#include <chrono>
#include <cstdio>
#include <thread>

using fa::StreamBlocks;
using fa::WorkspaceHold;

int main() {
    int a = 0, b = 0;  // two streams
    StreamBlocks blocks;
    // A call writes to its block at one launch and reads it at the next; in between
    // another thread may run.  Every call grows the block, as larger ones do.
    std::atomic<int> wrong{0}, calls{0};
    auto caller = [&](int id, void* stream, int n) {
        for (int i = 0; i < n; ++i) {
            WorkspaceHold hold = blocks.take(stream);
            hold->bytes = static_cast<std::size_t>(id);
            std::this_thread::yield();
            if (i % 16 == 0) std::this_thread::sleep_for(std::chrono::microseconds(50));
            if (hold->bytes != static_cast<std::size_t>(id) || hold->gone || hold->stream != stream)
                ++wrong;
            ++calls;
        }
    };
    std::thread t1(caller, 1, &a, 2000), t2(caller, 2, &a, 2000), t3(caller, 3, &b, 2000);
    std::size_t released = 0;
    while (calls < 6000) {
        for (auto& x : blocks.clear()) {
            if (!x->gone) ++wrong;
            ++released;
        }
        std::this_thread::sleep_for(std::chrono::milliseconds(1));
    }
    t1.join();
    t2.join();
    t3.join();
    if (wrong || !released) return std::printf("%d wrong\n", wrong.load()), 1;

    // the second call of a stream waits for the first; one of another stream does not
    std::atomic<bool> got{false};
    {
        WorkspaceHold first = blocks.take(&a);
        WorkspaceHold other = blocks.take(&b);
        std::thread second([&] {
            WorkspaceHold h = blocks.take(&a);
            got = true;
        });
        std::this_thread::sleep_for(std::chrono::milliseconds(100));
        if (got) return std::printf("not exclusive\n"), 2;
        {
            WorkspaceHold done = std::move(first);
        }
        second.join();
    }
    // a release waits for it too, and a later call gets a block of its own
    std::shared_ptr<fa::StreamBlock> old;
    std::atomic<bool> cleared{false};
    std::thread release;
    {
        WorkspaceHold h = blocks.take(&a);
        h->bytes = 77;
        release = std::thread([&] {
            for (auto& x : blocks.clear())
                if (x->bytes == 77) old = x;
            cleared = true;
        });
        std::this_thread::sleep_for(std::chrono::milliseconds(100));
        if (cleared) return std::printf("released in use\n"), 3;
    }
    release.join();
    if (!old || !old->gone) return std::printf("not released\n"), 4;
    if (blocks.take(&a)->bytes != 0) return std::printf("released block used\n"), 5;
    // what could not be freed comes again, and is nobody's meanwhile
    blocks.clear();
    blocks.keep(old);
    if (blocks.take(&a)->bytes != 0) return std::printf("kept block used\n"), 6;
    int again = 0;
    for (auto& x : blocks.clear()) again += x == old;
    if (again != 1 || !blocks.clear().empty()) return std::printf("kept block lost\n"), 7;
    std::printf("ok\n");
    return 0;
}
"""


def test_one_call_at_a_time_has_a_streams_workspace(tmp_path):
    src, exe = tmp_path / "harness.cpp", tmp_path / "harness"
    src.write_text(HARNESS)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-pthread", "-I",
                    os.path.join(fa_build.CSRC), str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert (out.returncode, out.stdout.strip()) == (0, "ok")

// Eight host threads set one flag's launch attributes at once: one of them runs
// the setter, and all read what it wrote behind the library's mutex.
#include <cstdarg>
#include <cstdio>
#include <thread>
#include <vector>

#include "tfq_internal.h"

namespace tfq {
std::mutex& state_mutex() {
    static std::mutex m;
    return m;
}
tfq_status fail(tfq_status st, const char*, ...) { return st; }
}  // namespace tfq

extern "C" const char* cudaGetErrorString(cudaError_t) { return ""; }  // no CUDA library is linked

int main() {
    for (int turn = 0; turn < 200; ++turn) {
        tfq::DeviceState ds;
        int set = 0, refused = 0;
        std::vector<std::thread> threads;
        std::vector<int> seen(8);
        for (int t = 0; t < 8; ++t)
            threads.emplace_back([&, t] {
                for (int i = 0; i < 4; ++i) {
                    const tfq_status st = tfq::once_per_device(ds.norm_attr_set, [&] {
                        if (++refused == 1) return cudaErrorInvalidValue;  // a failed attempt is made again
                        ++set;
                        return cudaSuccess;
                    });
                    if (st == TFQ_OK) seen[t] = set;
                }
            });
        for (auto& t : threads) t.join();
        for (int s : seen)
            if (s != 1 || set != 1 || refused != 2 || !ds.norm_attr_set) return 1;
    }
    std::puts("ok");
    return 0;
}

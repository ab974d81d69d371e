// The launches of paged_attention at the ends of the sizes that it accepts (test infrastructure, host only): the
// runtime's entry points are replaced by ones that record each launch's grid and run nothing, so no pointer is read.
// Every grid has fewer than 2^32 threads along x and no more than 65535 workgroups along y and z.  Prints "attention launches ok".
#include <algorithm>
#include <atomic>
#include <cstdio>
#include <cstring>
#include <map>
#include <string>
#include <vector>

#include <hip/hip_runtime.h>

#include "../../include/qgemm.h"
#include "launch.h"

struct Recorded {
    std::string kernel;
    dim3 grid, block;
};
static std::vector<Recorded> launches;
// (kernels are registered before main, perhaps before the objects of this file exist)
static std::map<const void*, std::string>& names() {
    static std::map<const void*, std::string> all;
    return all;
}
static dim3 pushed_grid, pushed_block;
static size_t pushed_lds;
static hipStream_t pushed_stream;

extern "C" {
char __hip_fatbin[64] = {0};
void** __hipRegisterFatBinary(const void*) {
    static void* handle;
    return &handle;
}
void __hipUnregisterFatBinary(void**) {}
void __hipRegisterFunction(void**, const void* host, char*, const char* device, unsigned, void*, void*, void*, void*, int*) {
    names()[host] = device;
}
hipError_t __hipPushCallConfiguration(dim3 grid, dim3 block, size_t lds, hipStream_t st) {
    pushed_grid = grid, pushed_block = block, pushed_lds = lds, pushed_stream = st;
    return hipSuccess;
}
hipError_t __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* lds, hipStream_t* st) {
    *grid = pushed_grid, *block = pushed_block, *lds = pushed_lds, *st = pushed_stream;
    return hipSuccess;
}
hipError_t hipLaunchKernel(const void* f, dim3 grid, dim3 block, void**, size_t, hipStream_t) {
    launches.push_back({names()[f], grid, block});
    return hipSuccess;
}
hipError_t hipGetLastError() { return hipSuccess; }
}
namespace qg {
int device_cu_count() { return 256; }
void allow_dynamic_lds(const void*, int, std::atomic<uint64_t>&) {}
void launch_qk_norm_rope(const RopeArgs&, int, hipStream_t) {}
void launch_kv_append(const RopeArgs&, int, hipStream_t) {}
}  // namespace qg

int main() {
    int failures = 0, calls = 0;
    long long most = 0;
    auto* p = reinterpret_cast<uint16_t*>(uintptr_t{1} << 20);
    auto* f = reinterpret_cast<float*>(p);
    auto* i = reinterpret_cast<int32_t*>(p);
    for (int Hkv : {1, 8, 64, 128, 512, 1024})
        for (int G : {1, 4, 16, 17, 64})
            for (int D : {64, 128})
                for (int B : {1, 2, 9, 500, 1 << 14, (1 << 23) / Hkv - 1})
                    for (long long tokens : {1LL, (long long)B, 17LL * B, 1LL << 40})
                        for (int prefix : {0, 256, 1 << 20})
                            for (int max_q : {0, 1, 17, 1 << 22})
                                for (float* scale : {static_cast<float*>(nullptr), f}) {
                                    const int Hq = Hkv * G, page = 256;
                                    if (Hq > 1024 || B > 1 << 14 || (long long)B * Hkv >= 1 << 23) continue;
                                    const long long T_most = std::min((1LL << 22) - 1, (1LL << 27) / Hq);
                                    const int T = (int)std::min(tokens, T_most), width = 1 << 14;
                                    launches.clear();
                                    const qg_status st = paged_attention(p, p, p, scale, scale, 1000, page, i, i, i, T, B, width, Hq,
                                                                         Hkv, D, 0.1f, 0, 0, prefix, max_q, p, f, p, ~size_t{0}, nullptr);
                                    ++calls;
                                    if (st != QG_OK || launches.empty()) {
                                        std::printf("status %d, %zu launches\n", st, launches.size());
                                        ++failures;
                                    }
                                    for (const Recorded& r : launches) {
                                        const long long x = (long long)r.grid.x * r.block.x;
                                        most = std::max(most, x);
                                        if (x < 1 || x >= 1LL << 32 || r.grid.y > 65535 || r.grid.z > 65535 || r.block.x != 256) {
                                            if (failures++ < 5)
                                                std::printf("%s: %u x %u x %u workgroups: T %d B %d Hq %d Hkv %d prefix %d max_q %d\n",
                                                            r.kernel.c_str(), r.grid.x, r.grid.y, r.grid.z, T, B, Hq, Hkv, prefix, max_q);
                                        }
                                    }
                                }
    std::printf("%d calls, %lld threads along x at most, %d failures\n", calls, most, failures);
    if (failures) return 1;
    std::puts("attention launches ok");
    return 0;
}

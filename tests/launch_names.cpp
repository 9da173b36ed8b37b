// Stands in for the HIP runtime's registration and launch calls (preloaded): no
// kernel runs; the names of the kernels that the library holds, and of those that
// a call launches, are kept.
#include <cstddef>
#include <map>
#include <string>
#include <vector>

namespace {
std::map<const void*, std::string>& held() {
    static std::map<const void*, std::string> names;
    return names;
}
std::vector<std::string> launched;
std::string joined;

const char* lines(const std::vector<std::string>& names) {
    joined.clear();
    for (const std::string& n : names) joined += n + "\n";
    return joined.c_str();
}
}  // namespace

struct Dim3 {
    unsigned x, y, z;
};

extern "C" {
// Names in lines; the memory is valid until the next of these calls.
const char* kernels_held() {
    std::vector<std::string> names;
    for (const auto& k : held()) names.push_back(k.second);
    return lines(names);
}
const char* kernels_launched() {
    const char* names = lines(launched);
    launched.clear();
    return names;
}

void** __hipRegisterFatBinary(const void*) {
    static void* module;
    return &module;
}
void __hipUnregisterFatBinary(void**) {}
void __hipRegisterVar(void**, void*, char*, char*, int, size_t, int, int) {}
void __hipRegisterFunction(void**, const void* stub, char*, const char* name, unsigned, void*, void*, void*, void*,
                           int*) {
    held()[stub] = name;
}
int __hipPushCallConfiguration(Dim3, Dim3, size_t, void*) { return 0; }
int __hipPopCallConfiguration(Dim3* grid, Dim3* block, size_t* lds, void** stream) {
    *grid = *block = {1, 1, 1};
    *lds = 0;
    *stream = nullptr;
    return 0;
}
int hipLaunchKernel(const void* stub, Dim3, Dim3, void**, size_t, void*) {
    launched.push_back(held()[stub]);
    return 0;
}
int hipGetLastError() { return 0; }
}

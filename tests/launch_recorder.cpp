// Runs entry points of the library on a machine without a GPU and prints which kernels they launch. The HIP calls that a
// launch consists of are defined here, in front of the runtime's own, so that nothing is ever launched.
//
//   launch_recorder <library>     then, a line each: <function> <1: with a workspace, 0> <the arguments' bytes in hex>
//
// prints for each line the status and the launches: "0 | name x y z | name x y z", grids in workgroups.
#include <cxxabi.h>
#include <dlfcn.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

#include <iostream>
#include <map>
#include <sstream>
#include <string>
#include <vector>

struct Dim3 {
  uint32_t x, y, z;
};
struct Configuration {
  Dim3 grid, block;
  size_t shared;
  void* stream;
};
static std::map<const void*, std::string>& names() {
  static std::map<const void*, std::string> m;
  return m;
}
static Configuration last;
static std::string launches;

extern "C" {
void** __hipRegisterFatBinary(const void*) {
  static void* handle;
  return &handle;
}
void __hipUnregisterFatBinary(void**) {}
void __hipRegisterFunction(void**, const void* host, char*, const char* name, unsigned, void*, void*, void*, void*, int*) { names()[host] = name; }
void __hipRegisterVar(void**, void*, char*, char*, int, size_t, int, int) {}
int __hipPushCallConfiguration(Dim3 grid, Dim3 block, size_t shared, void* stream) {
  last = Configuration{grid, block, shared, stream};
  return 0;
}
int __hipPopCallConfiguration(Dim3* grid, Dim3* block, size_t* shared, void** stream) {
  *grid = last.grid, *block = last.block, *shared = last.shared, *stream = last.stream;
  return 0;
}
int hipLaunchKernel(const void* host, Dim3 grid, Dim3, void**, size_t, void*) {
  int status = 0;
  char* plain = abi::__cxa_demangle(names()[host].c_str(), nullptr, nullptr, &status);
  std::string name = status == 0 ? plain : names()[host];
  free(plain);
  for (const char* cut : {"void ", "she::", "(anonymous namespace)::"})
    for (size_t at; (at = name.find(cut)) != std::string::npos;) name.erase(at, std::string(cut).size());
  name = name.substr(0, name.find('('));
  launches += " | " + name + " " + std::to_string(grid.x) + " " + std::to_string(grid.y) + " " + std::to_string(grid.z);
  return 0;
}
int hipGetLastError() { return 0; }
}

int main(int argc, char** argv) {
  void* lib = argc > 1 ? dlopen(argv[1], RTLD_NOW) : nullptr;
  if (!lib) {
    fprintf(stderr, "%s\n", argc > 1 ? dlerror() : "library?");
    return 1;
  }
  void* workspace = reinterpret_cast<void*>(uintptr_t(0x10000));
  for (std::string line; std::getline(std::cin, line);) {
    std::istringstream in(line);
    std::string function, hex;
    int with_workspace = 0;
    in >> function >> with_workspace >> hex;
    void* f = dlsym(lib, function.c_str());
    if (!f) return 2;
    std::vector<uint64_t> args(hex.size() / 16 + 2);
    for (size_t i = 0; i + 1 < hex.size(); i += 2) reinterpret_cast<uint8_t*>(args.data())[i / 2] = static_cast<uint8_t>(std::stoi(hex.substr(i, 2), nullptr, 16));
    launches.clear();
    const int code = with_workspace ? reinterpret_cast<int (*)(const void*, void*, size_t, void*)>(f)(args.data(), workspace, size_t(1) << 60, nullptr)
                                    : reinterpret_cast<int (*)(const void*, void*)>(f)(args.data(), nullptr);
    std::cout << code << launches << std::endl;
  }
  return 0;
}
